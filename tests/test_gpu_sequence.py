"""GPU parity of decay attention (sequence form, gradients, single tokens) and
LayerNorm (with statistics, gradients) against the float64 oracle.

Tolerances.  With u = 2^-24, a float32 sum of n products is off by at most
n u times the sum of their absolute values in any order; tensor-core
accumulation truncates, which doubles that.  A value of decay attention is a
dot product of D, a sum over the tokens of its block and D products with the
state, itself a sum over all T tokens: n <= 2 (2 D + 128 + T) + 16 operations,
scaled by the oracle's magnitude A (the sum of the absolute values of all
terms).  bfloat16 operands: the weighted products q.k, the state and (where no
state is an output) the decayed keys enter the tensor cores as two bfloat16
values each.  The first leaves less than 2^-8 of the value, half a step of
which is at most 2^-17: 1.5 * 2^-16 A for the three, below the 2 * 2^-16 A
allowed.  From 8192 (sequence, token, head) rows on, the products and the keys
enter as one value each, off by half a step: 2^-8 A for either, 2 * 2^-8 A for
both.  There the error as a whole is held tighter: roundings independent of
one another add in quadrature, so its 2-norm stays below 1.5 > sqrt(2) times
that of the output's own rounding (which an output made of exact products has).
The decays'
powers add |w n| u, at most 104 u before they vanish in float32.  The output's
own rounding is half a step: 2^-8 (bfloat16) of the value.
"""
import numpy as np
import pytest

from oracle import sequence as seq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def vk():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import linear_complexity_vision_b200 as vk
    vk.load_library()
    return vk


def _tdtype(dt):
    import torch
    return torch.float32 if dt == "f32" else torch.bfloat16


def _dev(a, dt="f32"):
    """A device tensor and the float64 values it holds."""
    import torch
    if a is None:
        return None, None
    t = torch.from_numpy(np.ascontiguousarray(a)).to(_tdtype(dt)).cuda()
    return t, t.double().cpu().numpy()


def _np(t):
    return t.detach().double().cpu().numpy()


def _check(name, got, want, mag, dt, n, lossy=True, rounded=False):
    """|got - want| <= half a step of the type + n u mag (+ the operands' types)."""
    got = _np(got)
    assert np.isfinite(got).all(), name
    step = 2.0 ** -8 if dt == "bf16" else U
    split = 2 * (2.0 ** -8 if rounded else 2.0 ** -16) if dt == "bf16" and lossy else 0.0
    tol = step * np.abs(want) + (n * U + split) * mag + 1e-37
    bad = np.abs(got - want) > tol
    assert not bad.any(), (name, int(bad.sum()), float(np.max(np.abs(got - want) / tol)))
    if rounded:
        import torch
        own = _np(torch.from_numpy(want).to(torch.bfloat16)) - want
        assert np.linalg.norm(got - want) <= 1.5 * np.linalg.norm(own), name


def _ops(D, T):
    return 2 * (2 * D + 128 + T) + 16 + 104


def _on_tcgen05(dt, T, D):
    """Heads of whole 16-byte vectors, bfloat16 ones up to 128 channels, float32
    ones of 33 to 64, of enough tokens; bfloat16 ones of other widths above 32
    are spread to such for more tokens."""
    if dt == "f32":
        return D % 4 == 0 and 32 < D <= 64 and T > 96
    if D % 8:
        return D > 32 and T > (64 if D <= 64 else 32)
    return T > (32 if D <= 32 else 16)


class Problem:
    def __init__(self, dt, B, T, H, D, seed=0, packed=False, state=True, lens=None, w=None, scale=None):
        import torch
        r = np.random.default_rng([seed, B, T, H, D])
        C = H * D
        self.dt, self.B, self.T, self.H, self.D = dt, B, T, H, D
        self.scale = float(np.float32(D ** -0.5 if scale is None else scale))
        if packed:
            qkv, qkvd = _dev(r.normal(size=(B, T, 3 * C)), dt)
            (self.q, self.k, self.v), (self.qd, self.kd, self.vd) = qkv.chunk(3, -1), np.split(qkvd, 3, -1)
        else:
            (self.q, self.qd), (self.k, self.kd), (self.v, self.vd) = (_dev(r.normal(size=(B, T, C)), dt) for _ in range(3))
        self.g, self.gd = _dev(r.normal(size=(B, T, C)), dt)
        self.w, self.wd = _dev(np.exp(r.uniform(-6, 0.5, H)) if w is None else np.full(H, w, float))
        self.s, self.sd = _dev(r.normal(size=(B, H, D, D)) if state else None)
        self.gs, self.gsd = _dev(r.normal(size=(B, H, D, D)) if state else None)
        self.rounded = dt == "bf16" and _on_tcgen05(dt, T, D) and B * T * H >= 8192
        self.lens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.lensd = lens

    def fwd(self, vk, **kw):
        return vk.decay_attn_fwd(self.q, self.k, self.v, self.w, self.H, self.scale, self.s, self.lens, **kw)

    def bwd(self, vk, **kw):
        return vk.decay_attn_bwd(self.q, self.k, self.v, self.w, self.H, self.g, self.scale, self.s, self.gs, self.lens, **kw)

    def check_fwd(self, out, last):
        want, S, mag, M = seq.decay_attn(self.qd, self.kd, self.vd, self.wd, self.H, self.scale, self.sd, self.lensd)
        n = _ops(self.D, self.T)
        _check("out", out, want, mag, self.dt, n, rounded=self.rounded)
        if last is not None:
            _check("state", last, S, M, "f32", n)

    def check_bwd(self, got):
        want, mag = seq.decay_attn_bwd(self.qd, self.kd, self.vd, self.wd, self.H, self.gd, self.scale, self.sd, self.gsd, self.lensd)
        n = _ops(self.D, self.T)
        for i, name in enumerate(("gq", "gk", "gv")):
            _check(name, got[i], want[i], mag[i], self.dt, n, rounded=self.rounded)
        if got[3] is not None:
            _check("gstate", got[3], want[3], mag[3], "f32", n)


CASES = [
    # dtype, B, T, H, D, packed, state, lengths
    ("bf16", 1, 1, 1, 64, False, True, None),
    ("bf16", 2, 2, 3, 64, False, False, None),
    ("bf16", 1, 31, 2, 64, True, True, None),
    ("bf16", 2, 127, 1, 64, False, True, None),
    ("bf16", 1, 128, 2, 64, True, False, None),
    ("bf16", 1, 129, 2, 64, False, True, None),
    ("bf16", 2, 196, 3, 64, True, True, None),
    ("bf16", 5, 300, 1, 64, True, True, [0, 1, 128, 300, 257]),
    ("bf16", 2, 40, 2, 64, False, True, [-3, 1000]),
    ("bf16", 1, 1500, 1, 64, False, True, None),          # cut into segments
    ("bf16", 3, 700, 1, 64, True, True, [700, 0, 390]),   # segments that a sequence does not reach
    ("bf16", 1, 5, 1, 128, False, True, None),
    ("bf16", 2, 196, 2, 128, True, True, None),
    ("bf16", 2, 260, 1, 128, False, False, [256, 131]),
    ("bf16", 1, 900, 1, 128, True, True, None),
    ("bf16", 1, 200, 2, 32, True, True, None),
    ("bf16", 2, 77, 3, 48, True, True, [77, 40]),
    ("bf16", 1, 130, 2, 9, False, True, None),
    ("bf16", 2, 33, 1, 1, False, True, None),
    ("f32", 1, 1, 2, 64, False, True, None),
    ("f32", 2, 33, 2, 64, True, True, None),
    ("f32", 3, 196, 2, 64, False, True, [196, 0, 65]),
    ("f32", 1, 1100, 1, 64, True, True, None),
    ("f32", 1, 150, 2, 128, True, True, None),
    ("f32", 2, 100, 2, 100, False, False, None),
    ("f32", 1, 64, 3, 7, False, True, None),
    ("f32", 2, 32, 1, 32, True, True, [31, 32]),
    ("bf16", 2, 150, 2, 8, True, True, [150, 20]),        # heads that are padded on their way in
    ("bf16", 1, 1300, 3, 24, True, True, None),
    ("bf16", 2, 200, 2, 72, True, True, [200, 90]),
    ("bf16", 1, 1100, 2, 120, False, True, None),
    ("f32", 2, 140, 3, 4, True, True, [140, 70]),
    ("f32", 1, 1100, 2, 36, True, True, None),
    ("f32", 3, 200, 1, 60, False, True, [200, 0, 131]),
    ("f32", 1, 300, 2, 66, True, True, None),
    ("bf16", 2, 300, 3, 5, True, True, [300, 77]),        # heads that are spread first
    ("bf16", 1, 1300, 2, 45, True, True, None),
    ("bf16", 3, 200, 2, 127, True, True, [200, 0, 131]),
    ("bf16", 1, 1000, 1, 67, False, True, None),
    ("f32", 1, 1100, 2, 37, True, True, None),
    ("f32", 3, 150, 2, 63, False, True, [150, 0, 131]),
]


def _kernel(dt, T, D):
    if not _on_tcgen05(dt, T, D):
        return "decay_attn_kernel"
    return "decay_attn_tcf_kernel" if dt == "f32" else "decay_attn_tc64_kernel" if D <= 64 else "decay_attn_tc_kernel"


@pytest.mark.parametrize("dt,B,T,H,D,packed,state,lens", CASES)
def test_forward(vk, dt, B, T, H, D, packed, state, lens):
    p = Problem(dt, B, T, H, D, 1, packed, state, lens)
    out, last = p.fwd(vk)
    vk.device_status()
    assert vk.load_library().vrwkv_last_kernel().decode() == _kernel(dt, T, D)
    p.check_fwd(out, last)
    again = p.fwd(vk)
    assert (again[0] == out).all() and (again[1] == last).all()
    only, none = p.fwd(vk, want_state=False)  # the tensor cores form a state that stays inside from fewer pieces
    assert none is None
    p.check_fwd(only, None)


@pytest.mark.parametrize("dt,B,T,H,D,packed,state,lens", CASES)
def test_backward(vk, dt, B, T, H, D, packed, state, lens):
    p = Problem(dt, B, T, H, D, 2, packed, state, lens)
    got = p.bwd(vk)
    vk.device_status()
    assert vk.load_library().vrwkv_last_kernel().decode() == _kernel(dt, T, D)
    p.check_bwd(got)
    again = p.bwd(vk)
    for a, b in zip(got, again):
        assert a is None or (a == b).all()


def test_any_size_kernel_on_tcgen05_sizes(vk, monkeypatch):
    """Heads of 64 and 128 channels whose rows start between 16-byte
    boundaries, and the same with the switch."""
    import torch
    for dt, D in (("bf16", 64), ("bf16", 128), ("f32", 64)):
        p = Problem(dt, 2, 300, 1, D, 14, lens=[300, 140])
        odd = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
        p.q, p.k, p.v, p.g = (odd(t) for t in (p.q, p.k, p.v, p.g))
        p.check_fwd(*p.fwd(vk))
        assert vk.load_library().vrwkv_last_kernel() == b"decay_attn_kernel"
        p.check_bwd(p.bwd(vk))
        monkeypatch.setenv("VRWKV_DECAY_TC", "0")
        p = Problem(dt, 1, 1000, 1, D, 15)
        p.check_fwd(*p.fwd(vk))
        assert vk.load_library().vrwkv_last_kernel() == b"decay_attn_kernel"
        p.check_bwd(p.bwd(vk))
        monkeypatch.delenv("VRWKV_DECAY_TC")


@pytest.mark.parametrize("dt,B,T,H", [("f32", 60, 150, 4), ("f32", 2, 700, 3), ("f32", 1, 2100, 1)])
def test_float32_heads_of_64(vk, dt, B, T, H):
    """Decays on either side of the factored path's bound, several blocks, cuts."""
    r = np.random.default_rng(18)
    p = Problem(dt, B, T, H, 64, 18, True, True, [int(x) for x in r.integers(0, T + 1, B - 1)] + [T],
                w=np.exp(np.linspace(-6, 0.3, H)))
    p.check_fwd(*p.fwd(vk))
    p.check_fwd(p.fwd(vk, want_state=False)[0], None)
    p.check_bwd(p.bwd(vk))
    vk.device_status()


@pytest.mark.parametrize("B,T,H,state,ragged", [(60, 150, 7, False, False), (40, 196, 5, True, True), (90, 20, 4, True, True),
                                                (25, 300, 8, False, True)])
def test_more_heads_than_sms(vk, B, T, H, state, ragged):
    """Several heads per persistent CTA, each head with a decay of its own on
    either side of the fast path's bound, sequences of any number of blocks."""
    lens = [int(x) for x in np.random.default_rng(16).integers(0, T + 1, B)] if ragged else None
    p = Problem("bf16", B, T, H, 64, 17, True, state, lens, w=np.exp(np.linspace(-6, 1, H)))
    out, last = p.fwd(vk)
    vk.device_status()
    p.check_fwd(out, last)
    p.check_fwd(p.fwd(vk, want_state=False)[0], None)
    got = p.bwd(vk)
    vk.device_status()
    p.check_bwd(got)


@pytest.mark.parametrize("B,T,H,lens", [(20, 300, 2, True), (2, 2100, 2, False)])
def test_heads_of_128(vk, B, T, H, lens):
    """From 8192 rows on, decays on either side of the factored path's bound."""
    r = np.random.default_rng(19)
    p = Problem("bf16", B, T, H, 128, 19, True, True, [int(x) for x in r.integers(0, T + 1, B)] if lens else None,
                w=np.exp(np.linspace(-4, 0.3, H)))
    assert p.rounded
    p.check_fwd(*p.fwd(vk))
    p.check_fwd(p.fwd(vk, want_state=False)[0], None)
    p.check_bwd(p.bwd(vk))
    vk.device_status()


@pytest.mark.parametrize("dt,B,T,H,D", [("bf16", 30, 300, 3, 40), ("bf16", 2, 2100, 2, 16), ("bf16", 25, 200, 5, 96),
                                        ("bf16", 1, 4200, 2, 88), ("bf16", 30, 150, 3, 33),
                                        ("bf16", 3, 1500, 2, 125), ("f32", 40, 150, 4, 50), ("f32", 40, 150, 4, 44), ("f32", 2, 1500, 2, 32)])
def test_padded_heads_and_their_neighbours(vk, dt, B, T, H, D):
    """Heads narrower than the tensor cores' tiles, several a CTA and cut: only
    their own channels are written, inside buffers whose rest keeps its values."""
    import torch
    r = np.random.default_rng([20, D])
    p = Problem(dt, B, T, H, D, 20, True, True, [int(x) for x in r.integers(0, T + 1, B - 1)] + [T],
                w=np.exp(np.linspace(-4, 0.3, H)))
    assert p.rounded == (dt == "bf16")
    n, ns = B * T * H * D, p.s.numel()
    buf, last = torch.full((n + 256,), 7.0, dtype=p.q.dtype, device="cuda"), torch.full((ns + 64,), 7.0, device="cuda")
    got = p.fwd(vk, out=buf[128:128 + n].view(B, T, H * D), state_out=last[32:32 + ns].view(p.s.shape))
    assert vk.load_library().vrwkv_last_kernel().decode() == _kernel(dt, T, D)
    p.check_fwd(*got)
    for b, m in ((buf, 128), (last, 32)):
        assert (b[:m] == 7).all() and (b[-m:] == 7).all()
    p.check_fwd(p.fwd(vk, want_state=False)[0], None)
    p.check_bwd(p.bwd(vk))
    vk.device_status()


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 20), ("bf16", 9)])
@pytest.mark.parametrize("T", [100, 1500])
def test_states_between_vector_boundaries(vk, dt, D, T):
    """States and their gradients that start 4 bytes past a 16-byte boundary."""
    import torch
    p = Problem(dt, 1, T, 1, D, 21)
    odd = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
    p.s, p.gs = odd(p.s), odd(p.gs)
    assert p.s.data_ptr() % 16 == 4
    p.check_fwd(*p.fwd(vk, state_out=odd(p.s)))
    p.check_bwd(p.bwd(vk))


@pytest.mark.parametrize("dt,D", [("f32", 64), ("f32", 9), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("scale", [0.0, 1e-30, -2.0, 1e15])
def test_scales(vk, dt, D, scale):
    """A scale of nothing, of no size that a state could carry, negative, large:
    the states do not depend on it."""
    p = Problem(dt, 2, 200, 2, D, 24, lens=[200, 65], scale=scale)
    out, last = p.fwd(vk)
    want, S, mag, M = seq.decay_attn(p.qd, p.kd, p.vd, p.wd, p.H, p.scale, p.sd, p.lensd)
    n = _ops(D, 200)
    _check("state", last, S, M, "f32", n)
    if abs(scale) != 1e-30:  # outputs below 1e-24 may lose bits
        _check("out", out, want, mag, dt, n)
        p.check_bwd(p.bwd(vk))
    else:
        assert np.isfinite(_np(out)).all()


def test_two_streams_at_once(vk):
    """Calls side by side on two streams, each with workspaces of its own."""
    import torch
    probs = [Problem("bf16", 1, 3000, 3, 64, 25), Problem("f32", 2, 900, 3, 64, 26), Problem("bf16", 1, 2000, 2, 128, 27),
             Problem("bf16", 2, 700, 3, 45, 28)]
    want = [(p.fwd(vk), p.bwd(vk)) for p in probs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in probs]
    spaces = [[vk.decay_attn_workspace(p.B, p.T, p.H, p.D, p.q.dtype, backward=b) for b in (False, True)] for p in probs]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got = []
        for p, s, (wf, wb) in zip(probs, streams, spaces):
            with torch.cuda.stream(s):
                got.append((p.fwd(vk, workspace=wf), p.bwd(vk, workspace=wb)))
    torch.cuda.synchronize()
    vk.device_status()
    for (wf, wb), (gf, gb) in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip((*wf, *wb), (*gf, *gb)))


def test_rows_and_states_far_apart(vk):
    """Rows whose offsets pass 32 bits, in elements, and a pool of states of
    more than 4 GiB."""
    import torch
    for dt, D in (("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 7)):
        ld, T = (1 << 33) // 520 // 16 * 16, 530
        p = Problem(dt, 1, T, 1, D, 22)
        far = torch.empty(ld * T, dtype=p.q.dtype, device="cuda")
        for i, name in enumerate("qkvg"):
            t = far.as_strided((1, T, D), (ld * T, ld, 1), i * D)
            t.copy_(getattr(p, name))
            setattr(p, name, t)
        p.check_fwd(*p.fwd(vk))
        p.check_bwd(p.bwd(vk))
        del far, t
        p.q = p.k = p.v = p.g = None
    N, D = 70000, 128
    pool = torch.empty((N, 1, D, D), device="cuda")
    slots = torch.tensor([N - 1, 0, 40000], dtype=torch.int32, device="cuda")
    p = Problem("bf16", 3, 1, 1, D, 23)
    pool[slots.long()] = p.s
    q, k, v = (t[:, 0].contiguous() for t in (p.q, p.k, p.v))
    out = vk.decay_attn_step(q, k, v, p.w, 1, pool, slots=slots, scale=p.scale)
    vk.device_status()
    p.check_fwd(out[:, None], pool[slots.long()])


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("f32", 64), ("bf16", 40)])
@pytest.mark.parametrize("w", [0.0, 0.7, 3.0, 1e4, float("inf"), -0.01])
def test_decays(vk, dt, D, w):
    """No decay, ordinary ones, ones that leave only the token itself, growth."""
    p = Problem(dt, 1, 150, 2, D, 3, w=w)
    if w == float("inf"):  # a state that no earlier token reaches
        p.wd = np.full(2, 1e6)
    p.check_fwd(*p.fwd(vk))
    p.check_bwd(p.bwd(vk))


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("f32", 64), ("bf16", 24), ("bf16", 45), ("f32", 44)])
def test_rows_past_the_end_are_not_used(vk, dt, D):
    """NaN and infinities behind the sequences' ends change no bit."""
    import torch
    B, T, H, lens = 3, 200, 2, [70, 0, 199]
    p = Problem(dt, B, T, H, D, 4, lens=lens)
    want_f, want_b = p.fwd(vk), p.bwd(vk)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(_tdtype(dt)).min], device="cuda").to(_tdtype(dt))
    for t in (p.q, p.k, p.v, p.g):
        for b, n in enumerate(lens):
            t[b, n:] = bad[torch.arange(t[b, n:].numel(), device="cuda") % 4].view(T - n, -1)
    for want, got in ((want_f, p.fwd(vk)), (want_b, p.bwd(vk))):
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_outputs_are_written_whole_and_only_they(vk):
    """Preallocated outputs inside larger buffers: the neighbours keep their
    values, the padded rows are zeros."""
    import torch
    for dt, D in (("bf16", 64), ("f32", 64), ("bf16", 20)):
        p = Problem(dt, 2, 150, 2, D, 5, lens=[150, 31])
        n = p.q.numel()
        buf = torch.full((n + 256,), 7.0, dtype=p.q.dtype, device="cuda")
        out = buf[128:128 + n].view(p.q.shape)
        got, last = p.fwd(vk, out=out)
        assert got.data_ptr() == out.data_ptr()
        assert (buf[:128] == 7).all() and (buf[128 + n:] == 7).all() and not got[1, 31:].any()
        p.check_fwd(got, last)


def test_state_in_place_and_pieces(vk):
    """A prompt in three pieces, its state updated in place, then single
    tokens: the same as the whole sequence."""
    import torch
    for dt, D, H in (("bf16", 64, 2), ("bf16", 128, 1), ("f32", 48, 2)):
        B, T = 2, 500
        p = Problem(dt, B, T, H, D, 6)
        state = p.s.clone()
        outs = []
        for a, b in ((0, 130), (130, 131), (131, 490)):
            q, k, v = (t[:, a:b].contiguous() for t in (p.q, p.k, p.v))
            o, last = vk.decay_attn_fwd(q, k, v, p.w, H, p.scale, state=state, state_out=state)
            assert last.data_ptr() == state.data_ptr()
            outs.append(o)
        pool = torch.zeros((4, H, D, D), device="cuda")
        slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
        pool[slots.long()] = state
        for t in range(490, T):
            outs.append(vk.decay_attn_step(p.q[:, t].contiguous(), p.k[:, t].contiguous(), p.v[:, t].contiguous(), p.w, H, pool,
                                           slots=slots, scale=p.scale)[:, None])
        vk.device_status()
        p.check_fwd(torch.cat(outs, 1), pool[slots.long()])
        assert not pool[0].any() and not pool[2].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,D", [(1, 1, 64), (3, 12, 64), (2, 3, 128), (5, 2, 32), (2, 2, 9), (1, 4, 1), (70, 2, 80)])
def test_step(vk, dt, B, H, D):
    import torch
    r = np.random.default_rng([7, B, H, D])
    N = B + 3
    x, xd = _dev(r.normal(size=(B, 3 * H * D)), dt)       # slices of one projection
    (q, k, v), (qd, kd, vd) = x.chunk(3, -1), np.split(xd, 3, -1)
    w, wd = _dev(np.exp(r.uniform(-6, 1, H)))
    s, sd = _dev(r.normal(size=(N, H, D, D)))
    slots = r.permutation(N)[:B]
    out = vk.decay_attn_step(q, k, v, w, H, s, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), scale=0.25)
    vk.device_status()
    want, pool, mag = seq.decay_attn_step(qd, kd, vd, wd, H, sd, slots, 0.25)
    _check("out", out, want, mag, dt, 2 * D + 16, lossy=False)
    M = np.abs(sd) + np.abs(pool)
    _check("state", s, pool, M, "f32", 8)
    used = np.isin(np.arange(N), slots)
    assert np.array_equal(_np(s)[~used], sd[~used])       # states that no row names
    s2, _ = _dev(sd[:B])
    got = vk.decay_attn_step(q, k, v, w, H, s2, scale=0.25)
    _check("no slots", got, *[seq.decay_attn_step(qd, kd, vd, wd, H, sd[:B], range(B), 0.25)[i] for i in (0, 2)], dt, 2 * D + 16, lossy=False)


def test_step_idle_repeated_and_bad_slots(vk):
    import torch
    H, D, N = 2, 64, 5
    r = np.random.default_rng(8)
    q, k, v = (_dev(r.normal(size=(6, H * D)))[0] for _ in range(3))
    qd, kd, vd = (_np(t) for t in (q, k, v))
    w, wd = _dev([0.1, 0.5])
    for slots, bad in (([2, -1, 0, -7, 4, 1], False), ([2, 2, 0, 2, 0, 1], True), ([5, 1, 1 << 30, -1, 0, 3], True)):
        s, sd = _dev(r.normal(size=(N, H, D, D)))
        out = vk.decay_attn_step(q, k, v, w, H, s, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
        want, pool, mag = seq.decay_attn_step(qd, kd, vd, wd, H, sd, slots)
        _check("out", out, want, mag, "f32", 2 * D + 16)
        _check("state", s, pool, np.abs(sd) + np.abs(pool), "f32", 8)
        for b, slot in enumerate(slots):
            if slot < 0 or slot >= N or slot in slots[:b]:
                assert not out[b].any()
        if bad:
            with pytest.raises(vk.VrwkvError, match="slot"):
                vk.device_status()
        vk.device_status()


def _ln_inputs(dt, rows, C, seed):
    r = np.random.default_rng([seed, rows, C])
    x, xd = _dev(r.normal(size=(rows, C)) * r.uniform(0.2, 3, (rows, 1)) + r.normal(size=(rows, 1)), dt)
    g, gd = _dev(r.normal(size=(rows, C)), dt)
    gamma, gammad = _dev(1 + 0.3 * r.normal(size=C))
    beta, betad = _dev(r.normal(size=C))
    return x, xd, g, gd, gamma, gammad, beta, betad


LN_CASES = [(1, 1), (3, 2), (5, 33), (40, 64), (7, 192), (1000, 96), (33, 384), (600, 768), (301, 1024), (9, 1030),
            (4, 2048), (6, 2056), (3, 4100), (5, 8192)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,C", LN_CASES)
def test_layer_norm(vk, dt, rows, C):
    x, xd, g, gd, gamma, gammad, beta, betad = _ln_inputs(dt, rows, C, 9)
    y, mean, rstd = vk.layer_norm_fwd(x, gamma, beta, 1e-5)
    yd, md, rd = seq.layer_norm_fwd(xd, gammad, betad, 1e-5)
    n = C + 16                                             # operations of a row's sums, in any order
    ax = np.abs(xd).mean(-1)
    dmean = n * U * ax                                     # how far the mean, then each term of the variance, is off
    assert (np.abs(_np(mean) - md) <= dmean + 1e-37).all()
    # rstd: half of the variance's relative error (its terms' errors come from
    # x - mean, and from the sum), and rsqrt's own two units
    var_off = n * U + 2 * (dmean + 2 * U * np.abs(xd).max(-1)) * rd + (dmean * rd) ** 2
    rel = 0.5 * var_off * 1.01 + 4 * U
    assert (np.abs(_np(rstd) - rd) <= rel * rd).all()
    step = 2.0 ** -8 if dt == "bf16" else U
    xh = (xd - md[:, None]) * rd[:, None]
    tol = (step * np.abs(yd) + np.abs(gammad) * (np.abs(xh) * (rel[:, None] + 4 * U) + rd[:, None] * (dmean[:, None] + U * np.abs(xd)))
           + 2 * U * (np.abs(betad) + np.abs(yd)))
    assert (np.abs(_np(y) - yd) <= tol * 1.01 + 1e-37).all()
    only = vk.layer_norm_fwd(x, gamma, beta, 1e-5, stats=False)
    assert only[1] is None and (only[0] == y).all()

    mean_d, rstd_d = _np(mean), _np(rstd)
    got = vk.layer_norm_bwd(x, gamma, mean, rstd, g)
    want, mag = seq.layer_norm_bwd(xd, gammad, mean_d, rstd_d, gd)
    # xh adds the rounding of x - mean, relative to x
    extra = 2 * U * rstd_d[:, None] * (np.abs(xd) + np.abs(mean_d)[:, None])
    d = np.abs(gammad * gd)
    slack = rstd_d[:, None] * (extra * (d * np.abs(xh)).mean(-1, keepdims=True) + np.abs(xh) * (d * extra).mean(-1, keepdims=True))
    assert (np.abs(_np(got[0]) - want[0]) <= step * np.abs(want[0]) + 1.01 * ((n + 16) * U * mag[0] + slack) + 1e-37).all()
    assert (np.abs(_np(got[1]) - want[1]) <= (rows + 16) * U * mag[1] + 1.01 * (np.abs(gd) * extra).sum(0) + 1e-37).all()
    assert (np.abs(_np(got[2]) - want[2]) <= (rows + 16) * U * mag[2] + 1e-37).all()
    again = vk.layer_norm_bwd(x, gamma, mean, rstd, g)
    assert all((a == b).all() for a, b in zip(got, again))
    bare = vk.layer_norm_bwd(x, gamma, mean, rstd, g, weight_grads=False)
    assert bare[1] is None and (bare[0] == got[0]).all()


def test_layer_norm_unaligned_rows(vk):
    """Tensors that start between two 16-byte boundaries, and rows without variance."""
    import torch
    for dt in ("bf16", "f32"):
        x, xd, g, gd, gamma, gammad, beta, betad = _ln_inputs(dt, 20, 64, 10)
        shift = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
        xs, gs, gms = shift(x), shift(g), shift(gamma)
        a, b = vk.layer_norm_fwd(x, gamma, beta), vk.layer_norm_fwd(xs, gms, shift(beta))
        yd, md, rd = seq.layer_norm_fwd(xd, gammad, betad, 1e-5)
        for got in (a, b):  # the two kernels' sums differ in order alone
            assert np.allclose(_np(got[0]), yd, rtol=2.0 ** -8 if dt == "bf16" else 1e-5, atol=1e-5)
        u, v = vk.layer_norm_bwd(x, gamma, a[1], a[2], g), vk.layer_norm_bwd(xs, gms, a[1], a[2], gs)
        want, mag = seq.layer_norm_bwd(xd, gammad, _np(a[1]), _np(a[2]), gd)
        for got in (u, v):
            assert (np.abs(_np(got[0]) - want[0]) <= (2.0 ** -8 if dt == "bf16" else U) * np.abs(want[0]) + 200 * U * (mag[0] + 4)).all()
    flat = torch.full((3, 64), 2.5, device="cuda")
    y, mean, rstd = vk.layer_norm_fwd(flat, gamma, beta, 1e-5)
    assert (y == beta).all() and (mean == 2.5).all()
    assert np.allclose(_np(rstd), 1e-5 ** -0.5, rtol=1e-6)
    gx, _, _ = vk.layer_norm_bwd(flat, gamma, mean, rstd, torch.ones_like(flat))
    assert np.isfinite(_np(gx)).all()


def test_streams_graphs_and_workspaces(vk):
    """Calls on a side stream, and captured and replayed ones, on their own
    workspaces, give the default stream's bits."""
    import torch
    p = Problem("bf16", 1, 1500, 2, 64, 11)
    f = Problem("f32", 2, 300, 2, 48, 12, lens=[300, 100])
    odd = Problem("bf16", 2, 1300, 2, 61, 29, lens=[1300, 700])
    gamma, beta = torch.ones(128, device="cuda"), torch.zeros(128, device="cuda")

    def calls(p):
        ws = vk.decay_attn_workspace(p.B, p.T, p.H, p.D, p.q.dtype)
        wb = vk.decay_attn_workspace(p.B, p.T, p.H, p.D, p.q.dtype, backward=True)
        x = p.q.contiguous().view(-1, p.D)
        wl = vk.layer_norm_bwd_workspace(x.shape[0], p.D, x.dtype)
        pool = p.s.clone()

        def run():
            out, last = p.fwd(vk, workspace=ws)
            grads = p.bwd(vk, workspace=wb)
            y, mean, rstd = vk.layer_norm_fwd(x, gamma[:p.D], beta[:p.D])
            ln = vk.layer_norm_bwd(x, gamma[:p.D], mean, rstd, x, workspace=wl)
            pool.copy_(p.s)
            o = vk.decay_attn_step(p.q[:, 0].contiguous(), p.k[:, 0].contiguous(), p.v[:, 0].contiguous(), p.w, p.H, pool)
            return [out, last, *grads, y, mean, rstd, *ln, o, pool]
        return run

    for prob in (p, f, odd):
        want = [t.clone() for t in calls(prob)()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run = calls(prob)
            got = run()
            for _ in range(2):
                run()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            captured = run()
        for t in captured:
            t.zero_()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, captured))
    vk.device_status()


def test_a_layer_forward_backward_and_decoding(vk):
    """LayerNorm -> q, k, v projections -> decay attention -> LayerNorm, its
    gradients against torch's float64 autograd of the formulas, and the same
    layer one token at a time.  float32: the projections (torch matmuls) and
    the operators are off by a few hundred u of their magnitudes."""
    import torch
    B, T, H, D = 2, 70, 2, 64
    C = H * D
    torch.manual_seed(13)
    x = torch.randn(B, T, C, device="cuda")
    W = torch.randn(C, 3 * C, device="cuda") / C ** 0.5
    ga, be, go, bo = (torch.randn(C, device="cuda") for _ in range(4))
    w = torch.tensor([0.05, 0.4], device="cuda")
    gy = torch.randn(B, T, C, device="cuda")
    # forward, keeping what the backward pass needs
    n1, m1, r1 = vk.layer_norm_fwd(x, ga, be)
    q, k, v = (n1 @ W).chunk(3, -1)
    a, last = vk.decay_attn_fwd(q, k, v, w, H, D ** -0.5)
    y, m2, r2 = vk.layer_norm_fwd(a, go, bo)
    # backward
    d_a, d_go, d_bo = vk.layer_norm_bwd(a, go, m2, r2, gy)
    d_qkv = torch.cat(vk.decay_attn_bwd(q, k, v, w, H, d_a, D ** -0.5)[:3], -1)
    d_W = n1.flatten(0, 1).T @ d_qkv.flatten(0, 1)
    d_x, d_ga, d_be = vk.layer_norm_bwd(x, ga, m1, r1, d_qkv @ W.T)

    def ln(x, g, b):
        mean = x.mean(-1, keepdim=True)
        return (x - mean) / ((x - mean).square().mean(-1, keepdim=True) + 1e-5).sqrt() * g + b

    ps = [t.double().requires_grad_() for t in (x, W, ga, be, go, bo)]
    qd, kd, vd = (t.view(B, T, H, D).transpose(1, 2) for t in (ln(ps[0], ps[2], ps[3]) @ ps[1]).chunk(3, -1))
    i = torch.arange(T, device="cuda")
    dec = torch.tril(torch.exp(-w.double()[:, None, None] * (i[:, None] - i[None, :]).clamp(min=0)))
    ad = ((qd @ kd.transpose(-1, -2)) * dec * D ** -0.5) @ vd
    yd = ln(ad.transpose(1, 2).reshape(B, T, C), ps[4], ps[5])
    yd.backward(gy.double())
    for name, got, want in (("y", y, yd), ("x", d_x, ps[0].grad), ("W", d_W, ps[1].grad), ("ga", d_ga, ps[2].grad),
                            ("be", d_be, ps[3].grad), ("go", d_go, ps[4].grad), ("bo", d_bo, ps[5].grad)):
        off = float((got.detach().double() - want.detach()).norm() / want.detach().norm())
        assert off < 1e-5, (name, off)
    # decoding: one token at a time
    pool = torch.zeros(B, H, D, D, device="cuda")
    for t in range(T):
        n, _, _ = vk.layer_norm_fwd(x[:, t].contiguous(), ga, be, stats=False)
        o = vk.decay_attn_step(*(n @ W).chunk(3, -1), w, H, pool, scale=D ** -0.5)
        o, _, _ = vk.layer_norm_fwd(o, go, bo, stats=False)
        want = yd[:, t].detach()
        assert float((o.double() - want).norm() / want.norm()) < 1e-5
    assert float((pool - last).norm() / last.norm()) < 1e-5
    vk.device_status()
