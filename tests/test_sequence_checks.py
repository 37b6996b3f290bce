"""Refusals of decay attention and LayerNorm, on the host: the C ABI's checks
on stand-in pointers and the binding's on stand-in tensors.  No GPU is
touched: validation precedes every CUDA call."""
import ctypes

import pytest
import torch

import linear_complexity_vision_b200 as vk
from test_binding_checks import FakeCuda

M = 1 << 26
P = [M * (i + 1) for i in range(16)]  # non-null, 64 MiB apart, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from linear_complexity_vision_b200 import build
    build.build()
    return vk.load_library()


def _call(fn, names, defaults, args):
    a = dict(defaults, **args)
    return fn(*[a[n] for n in names.split()])


FWD = "q k v ldq ldk ldv w state lengths scale out state_out B T H D dtype ws ws_bytes stream"
FWD_OK = dict(q=P[0], k=P[1], v=P[2], ldq=256, ldk=256, ldv=256, w=P[3], state=None, lengths=None, scale=1.0, out=P[4],
              state_out=None, B=2, T=100, H=4, D=64, dtype=1, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("args,code,frag", [
    (dict(B=0), 1, "positive"),
    (dict(T=-1), 1, "positive"),
    (dict(H=0), 1, "positive"),
    (dict(D=0), 1, "positive"),
    (dict(D=129, ldq=1024, ldk=1024, ldv=1024), 2, "exceeds 128"),
    (dict(B=1 << 16, T=1 << 15), 2, "2^31"),
    (dict(dtype=3), 1, "dtype"),
    (dict(q=None), 1, "NULL"),
    (dict(w=None), 1, "NULL"),
    (dict(out=None), 1, "NULL"),
    (dict(ldk=255), 1, "row stride"),
    (dict(v=P[2] + 1), 1, "misaligned"),
    (dict(state=P[5] + 2), 1, "misaligned"),
    (dict(lengths=P[5] + 1), 1, "misaligned"),
    (dict(out=P[0] + 64), 1, "overlaps"),
    (dict(q=P[4] - 256, ldq=768), 1, "overlaps"),       # a strided input's span reaches the output
    (dict(state=P[5], state_out=P[5] + 4), 1, "overlaps"),
    (dict(state_out=P[4] + 4), 1, "overlap"),
    (dict(T=100000, B=1), 1, "workspace"),
    (dict(T=100000, B=1, ws=P[6] + 16, ws_bytes=1 << 24), 1, "256-byte"),
    (dict(T=100000, B=1, ws=P[6], ws_bytes=64), 1, "smaller"),
])
def test_decay_attn_fwd_rejects(lib, args, code, frag):
    assert _call(lib.vrwkv_decay_attn_fwd, FWD, FWD_OK, args) == code
    assert frag in lib.vrwkv_last_error().decode()


BWD = "q k v gy ldq ldk ldv ldg w state gstate lengths scale gq gk gv gs B T H D dtype ws ws_bytes stream"
BWD_OK = dict(q=P[0], k=P[1], v=P[2], gy=P[3], ldq=256, ldk=256, ldv=256, ldg=256, w=P[4], state=None, gstate=None,
              lengths=None, scale=1.0, gq=P[5], gk=P[6], gv=P[7], gs=None, B=2, T=100, H=4, D=64, dtype=1, ws=None,
              ws_bytes=0, stream=None)


@pytest.mark.parametrize("args,code,frag", [
    (dict(T=0), 1, "positive"),
    (dict(D=200, ldq=1024, ldk=1024, ldv=1024, ldg=1024), 2, "exceeds 128"),
    (dict(dtype=-1), 1, "dtype"),
    (dict(gy=None), 1, "NULL"),
    (dict(gv=None), 1, "NULL"),
    (dict(ldg=0), 1, "row stride"),
    (dict(gk=P[6] + 1), 1, "misaligned"),
    (dict(gs=P[8] + 1), 1, "misaligned"),
    (dict(gq=P[3]), 1, "overlaps"),
    (dict(gk=P[5] + 4096), 1, "overlap"),
    (dict(gstate=P[8], gs=P[8]), 1, "overlaps"),
    (dict(T=100000, B=1), 1, "workspace"),
])
def test_decay_attn_bwd_rejects(lib, args, code, frag):
    assert _call(lib.vrwkv_decay_attn_bwd, BWD, BWD_OK, args) == code
    assert frag in lib.vrwkv_last_error().decode()


STEP = "q k v ldq ldk ldv w state slots scale out B N H D dtype stream"
STEP_OK = dict(q=P[0], k=P[1], v=P[2], ldq=256, ldk=256, ldv=256, w=P[3], state=P[4], slots=None, scale=1.0, out=P[5],
               B=2, N=2, H=4, D=64, dtype=0, stream=None)


@pytest.mark.parametrize("args,code,frag", [
    (dict(B=0), 1, "positive"),
    (dict(N=0), 1, "at least one"),
    (dict(N=1), 1, "without slots"),
    (dict(D=129, ldq=1024, ldk=1024, ldv=1024), 2, "exceeds 128"),
    (dict(H=65536, D=1, ldq=1 << 17, ldk=1 << 17, ldv=1 << 17), 2, "65535"),
    (dict(state=None), 1, "NULL"),
    (dict(ldv=255), 1, "row stride"),
    (dict(k=P[1] + 2), 1, "misaligned"),
    (dict(slots=P[6] + 2), 1, "misaligned"),
    (dict(out=P[4] + 1024), 1, "overlap"),
    (dict(slots=P[4] + 4), 1, "overlaps"),
])
def test_decay_attn_step_rejects(lib, args, code, frag):
    assert _call(lib.vrwkv_decay_attn_step, STEP, STEP_OK, args) == code
    assert frag in lib.vrwkv_last_error().decode()


LNF = "x gamma beta eps y mean rstd rows C dtype stream"
LNF_OK = dict(x=P[0], gamma=P[1], beta=P[2], eps=1e-5, y=P[3], mean=P[4], rstd=P[5], rows=10, C=64, dtype=1, stream=None)


@pytest.mark.parametrize("args,code,frag", [
    (dict(rows=0), 1, "positive"),
    (dict(C=-4), 1, "positive"),
    (dict(rows=1 << 31), 2, "2^31"),
    (dict(dtype=2), 1, "dtype"),
    (dict(beta=None), 1, "NULL"),
    (dict(rstd=None), 1, "together"),
    (dict(eps=-1.0), 1, "eps"),
    (dict(eps=float("nan")), 1, "eps"),
    (dict(y=P[3] + 1), 1, "misaligned"),
    (dict(mean=P[4] + 2), 1, "misaligned"),
    (dict(y=P[0] + 128), 1, "overlaps"),
    (dict(mean=P[3] + 4), 1, "overlap"),
])
def test_layer_norm_fwd_rejects(lib, args, code, frag):
    assert _call(lib.vrwkv_layer_norm_fwd, LNF, LNF_OK, args) == code
    assert frag in lib.vrwkv_last_error().decode()


LNB = "x gamma mean rstd gy gx ggamma gbeta rows C dtype ws ws_bytes stream"
LNB_OK = dict(x=P[0], gamma=P[1], mean=P[2], rstd=P[3], gy=P[4], gx=P[5], ggamma=P[6], gbeta=P[7], rows=10, C=64, dtype=1,
              ws=P[8], ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("args,code,frag", [
    (dict(rows=-1), 1, "positive"),
    (dict(C=8193), 2, "exceeds 8192"),
    (dict(dtype=9), 1, "dtype"),
    (dict(gx=None), 1, "NULL"),
    (dict(gbeta=None), 1, "together"),
    (dict(gy=P[4] + 1), 1, "misaligned"),
    (dict(ws=None), 1, "workspace"),
    (dict(ws=P[8] + 128), 1, "256-byte"),
    (dict(ws_bytes=100), 1, "smaller"),
    (dict(gx=P[4]), 1, "overlaps"),
    (dict(ggamma=P[8] + 256), 1, "overlap"),
])
def test_layer_norm_bwd_rejects(lib, args, code, frag):
    assert _call(lib.vrwkv_layer_norm_bwd, LNB, LNB_OK, args) == code
    assert frag in lib.vrwkv_last_error().decode()


def test_workspace_sizes(lib):
    size = lib.vrwkv_decay_attn_workspace_bytes
    assert size(2, 100, 4, 64, 1, 0) == 0             # one segment: no cuts
    assert size(1, 100000, 1, 64, 1, 0) > 0
    assert size(1, 100000, 1, 64, 1, 1) > 0
    # heads that are spread: copies of three inputs and an output, or of four and three
    assert size(64, 200, 16, 45, 1, 0) == 4 * 64 * 200 * 16 * 48 * 2
    assert size(64, 200, 16, 45, 1, 1) == 7 * 64 * 200 * 16 * 48 * 2
    assert size(64, 200, 16, 45, 0, 0) == 0 and size(64, 60, 16, 45, 1, 0) == 0
    assert size(0, 100, 4, 64, 1, 0) == 0 and size(2, 100, 4, 129, 1, 0) == 0
    assert lib.vrwkv_layer_norm_bwd_workspace_bytes(10, 64, 1) >= 2 * 64 * 4
    assert lib.vrwkv_layer_norm_bwd_workspace_bytes(10, 8193, 1) == 0


def test_layer_norm_bwd_partial_rows(lib):
    """Widths that the same kernel serves get the same number of CTAs, each with a
    partial row of 2 C floats: as many as stay on an SM at a time."""
    rows = 1 << 20

    def ctas(C):
        n = lib.vrwkv_layer_norm_bwd_workspace_bytes(rows, C, 0)
        return n // (8 * C)                              # bytes are rounded up to 256, less than a row
    assert ctas(516) == ctas(640) == ctas(768)           # 6 vectors a lane
    assert ctas(772) == ctas(896) == ctas(1024)          # 8
    assert ctas(512) >= ctas(768) >= ctas(1024)


# ---- the binding ----


vk._load_torch()


class Rows(FakeCuda):
    """A stand-in with strides."""

    def __init__(self, shape, stride, **kw):
        super().__init__(shape, contiguous=False, **kw)
        self._stride = stride

    def stride(self):
        return self._stride


DEV = torch.device("cuda:0")


@pytest.mark.parametrize("shape,stride,ld", [
    ((2, 5, 8), (120, 24, 1), 24),      # a slice of a (2, 5, 24) projection
    ((1, 5, 8), (7, 24, 1), 24),        # one sequence: the batch stride has no meaning
    ((3, 1, 8), (24, 8, 1), 24),        # one token: rows are the sequences
    ((1, 1, 8), (9, 9, 1), 8),
    ((4, 8), (16, 1), 16),
])
def test_row_strides(shape, stride, ld):
    assert vk._require_rows("q", Rows(shape, stride), shape, torch.bfloat16, DEV) == ld


@pytest.mark.parametrize("shape,stride,msg", [
    ((2, 5, 8), (60, 8, 1), "evenly"),      # x[:, :5] of a longer batch
    ((2, 5, 8), (40, 1, 5), "adjacent"),    # transposed
    ((2, 5, 8), (0, 8, 1), "evenly"),       # an expanded batch
    ((2, 5, 8), (0, 0, 1), "overlap"),      # an expanded row
    ((2, 5, 8), (20, 4, 1), "overlap"),
])
def test_uneven_rows_are_refused(shape, stride, msg):
    with pytest.raises(ValueError, match=msg):
        vk._require_rows("q", Rows(shape, stride), shape, torch.bfloat16, DEV)


B, T, H, D = 2, 9, 4, 16
C = H * D


def tok(**kw):
    return FakeCuda((B, T, C), **kw)


def f32(*shape, **kw):
    return FakeCuda(shape, dtype=torch.float32, **kw)


@pytest.mark.parametrize("change,msg", [
    (dict(k=FakeCuda((B, T + 1, C))), "k must be"),
    (dict(v=FakeCuda((B, T, C), dtype=torch.float32)), "v must be"),
    (dict(k=FakeCuda((B, T, C), device="cuda:1")), "k must be a CUDA tensor on"),
    (dict(w=f32(H + 1)), "w must be"),
    (dict(heads=5), "whole number"),
    (dict(heads=0), "whole number"),
    (dict(state=f32(B, H, D, D + 1)), "state must be"),
    (dict(state=FakeCuda((B, H, D, D))), "state must be a float32"),
    (dict(state_out=f32(B + 1, H, D, D)), "state_out must be"),
    (dict(lengths=FakeCuda((B,), dtype=torch.int64)), "lengths must be an int32"),
    (dict(lengths=FakeCuda((B + 1,), dtype=torch.int32)), "lengths must be an int32"),
    (dict(out=FakeCuda((B, T, C + 4))), "out must match"),
])
def test_decay_attn_fwd_binding_refuses(change, msg):
    a = dict(q=tok(), k=tok(), v=tok(), w=f32(H), heads=H)
    a.update(change)
    with pytest.raises(ValueError, match=msg):
        vk.decay_attn_fwd(**a)


def test_decay_attn_bwd_binding_refuses():
    ok = dict(q=tok(), k=tok(), v=tok(), w=f32(H), heads=H, gy=tok(), out=(tok(), tok(), tok(), None))
    for change, msg in ((dict(gy=FakeCuda((B, T, C - 1))), "gy must be"), (dict(gstate=f32(B, H, D)), "gstate must be"),
                        (dict(out=(tok(), tok(), FakeCuda((B, C)), None)), "gv must match"),
                        (dict(out=(tok(), tok(), tok(), f32(1))), "gstate_in must be")):
        with pytest.raises(ValueError, match=msg):
            vk.decay_attn_bwd(**{**ok, **change})


def test_decay_attn_step_binding_refuses():
    row = FakeCuda((B, C))
    ok = dict(q=row, k=row, v=row, w=f32(H), heads=H, state=f32(5, H, D, D))
    for change, msg in ((dict(q=tok()), "q must be a"), (dict(k=FakeCuda((B, C + 1))), "k must be"),
                        (dict(state=f32(5, H, D)), "state must be"), (dict(state=f32(5, H, D, D, contiguous=False)), "contiguous"),
                        (dict(slots=FakeCuda((B,), dtype=torch.int64)), "slots must be an int32"),
                        (dict(out=FakeCuda((B, C), dtype=torch.float32)), "out must match")):
        with pytest.raises(ValueError, match=msg):
            vk.decay_attn_step(**{**ok, **change})


def test_layer_norm_binding_refuses():
    x = tok()
    with pytest.raises(ValueError, match="gamma must be"):
        vk.layer_norm_fwd(x, f32(C + 1), f32(C))
    with pytest.raises(ValueError, match="x must be a contiguous CUDA"):
        vk.layer_norm_fwd(FakeCuda((B, T, C), contiguous=False), f32(C), f32(C))
    with pytest.raises(ValueError, match="out must match"):
        vk.layer_norm_fwd(x, f32(C), f32(C), out=FakeCuda((B, C)))
    with pytest.raises(ValueError, match="with rows"):
        vk.layer_norm_fwd(FakeCuda((0, C)), f32(C), f32(C))
    with pytest.raises(ValueError, match="rstd must be"):
        vk.layer_norm_bwd(x, f32(C), f32(B, T), f32(B, T + 1), x)
    with pytest.raises(ValueError, match="gy must match"):
        vk.layer_norm_bwd(x, f32(C), f32(B, T), f32(B, T), FakeCuda((B, T, C), dtype=torch.float32), out=tok())


def test_argument_types_cover_every_entry_point(lib):
    for name in ("vrwkv_decay_attn_fwd", "vrwkv_decay_attn_bwd", "vrwkv_decay_attn_step", "vrwkv_layer_norm_fwd",
                 "vrwkv_layer_norm_bwd"):
        assert getattr(lib, name).argtypes is not None and getattr(lib, name).restype is ctypes.c_int


def test_remembered_workspace_sizes_are_bounded(monkeypatch):
    """A program whose sequences are of ever new lengths does not grow by them."""
    monkeypatch.setattr(vk, "_ws_need", {})
    asked = []
    for n in range(3 * vk._WS_NEED_MOST):
        def size():
            asked.append(n)
            return 0
        for _ in range(2):
            assert vk._workspace((1, n), size, None, DEV, None) == (None, 0, None)
    assert len(vk._ws_need) <= vk._WS_NEED_MOST
    assert asked == list(range(3 * vk._WS_NEED_MOST))  # once each while it is remembered


@pytest.mark.parametrize("T", [(1 << 30) + 1, (1 << 31) - 1])
def test_longest_sequences(lib, T):
    """Beyond 2^30 tokens the end of a segment, rounded up, would not be an int."""
    for fn, names, ok in ((lib.vrwkv_decay_attn_fwd, FWD, FWD_OK), (lib.vrwkv_decay_attn_bwd, BWD, BWD_OK)):
        assert _call(fn, names, ok, dict(B=1, T=T)) == 2
        assert "2^30" in lib.vrwkv_last_error().decode()
    assert lib.vrwkv_decay_attn_workspace_bytes(1, T, 1, 1, 1, 0) == 0


@pytest.mark.parametrize("C", [(1 << 30) + 1, (1 << 31) - 1])
def test_widest_rows(lib, C):
    """Beyond 2^30 channels a lane's next one, 32 on, might not be an int."""
    assert _call(lib.vrwkv_layer_norm_fwd, LNF, LNF_OK, dict(rows=1, C=C)) == 2
    assert "2^30" in lib.vrwkv_last_error().decode()


def test_sizes_that_are_no_c_int_are_refused():
    """ctypes cuts a C int off without a word: 2^32 + 5 tokens would be 5."""
    for n in (1 << 31, (1 << 32) + 5):
        x = FakeCuda((1, n, 4))
        with pytest.raises(ValueError, match="2\\^31"):
            vk.decay_attn_fwd(x, x, x, f32(1), 1)
        with pytest.raises(ValueError, match="2\\^31"):
            vk.decay_attn_bwd(x, x, x, f32(1), 1, x)
        row = FakeCuda((1, 4))
        with pytest.raises(ValueError, match="2\\^31"):
            vk.decay_attn_step(row, row, row, f32(1), 1, f32(n, 1, 4, 4))
        with pytest.raises(ValueError, match="2\\^31"):
            vk.layer_norm_fwd(FakeCuda((1, n)), f32(n), f32(n))
        with pytest.raises(ValueError, match="2\\^31"):
            vk.layer_norm_bwd(FakeCuda((1, n)), f32(n), f32(1), f32(1), FakeCuda((1, n)))
