"""The measured cases of the multi-head decay attention and LayerNorm operators.

Decay attention is causal linear attention whose state decays at a fixed rate
per head.  With the heads' channels side by side in C = H * D, tokens t, s and
a decay w_h of head h:

    out_t   = scale * q_t S_t,      S_t = e^{-w_h} S_{t-1} + k_t^T v_t
            = scale * [ sum_{s <= t} e^{-w_h (t - s)} (q_t . k_s) v_s + e^{-w_h (t + 1)} q_t S_{-1} ]

`fwd` is its form for prompts, `bwd` its gradient, `step` its form for single
tokens, which updates a pool of states in place.  `ln_fwd` and `ln_bwd` are
LayerNorm over channels with its statistics, and its gradient.

Every operator has a plain form in elementary torch operations and a float64
form (`exact`) that follows the recurrence token by token.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one 14 x 14 image's tokens as a prompt, three heads: a call that is all latency
        dict(name="fwd bf16 1x196x192", op="fwd", dtype="bf16", B=1, T=196, H=3, D=64, packed=False, lens=False, state=False, want=True),
        # a padded batch of 14 x 14 prompts in float32, each of its own length, continued from earlier states
        dict(name="fwd f32 32x196x384 ragged", op="fwd", dtype="f32", B=32, T=196, H=6, D=64, packed=False, lens=True, state=True, want=True),
        # the 64 x 64 grid at the benchmark's batch and width: a training step's forward
        dict(name="fwd bf16 8x4096x1024", op="fwd", dtype="bf16", B=8, T=4096, H=16, D=64, packed=False, lens=False, state=False, want=False),
        # the 16384 tokens of a 2048^2 image (patch 16) as one long prompt, 128 channels a head, its state kept for decoding
        dict(name="fwd bf16 1x16384x1024 D=128", op="fwd", dtype="bf16", B=1, T=16384, H=8, D=128, packed=False, lens=False, state=True, want=True),
        # training on 14 x 14 grids: many short sequences, q, k, v slices of one projection
        dict(name="bwd bf16 64x196x768", op="bwd", dtype="bf16", B=64, T=196, H=12, D=64, packed=True, lens=False, state=False),
        # training at the benchmark's shape
        dict(name="bwd bf16 8x4096x1024", op="bwd", dtype="bf16", B=8, T=4096, H=16, D=64, packed=False, lens=False, state=False),
        # float32 training on padded sequences of odd length, with the gradient of the state they start from
        dict(name="bwd f32 3x1001x384 ragged", op="bwd", dtype="f32", B=3, T=1001, H=6, D=64, packed=False, lens=True, state=True),
        # decoding one sequence: a call that is all latency
        dict(name="step bf16 1x768", op="step", dtype="bf16", B=1, H=12, D=64, pool=4),
        # decoding a full batch out of a pool of states
        dict(name="step bf16 256x1024", op="step", dtype="bf16", B=256, H=16, D=64, pool=300),
        # the norm after an output projection on 14 x 14 grids
        dict(name="ln_fwd bf16 12544x768", op="ln_fwd", dtype="bf16", rows=64 * 196, C=768),
        # its gradient in float32 at a narrow width
        dict(name="ln_bwd f32 6272x384", op="ln_bwd", dtype="f32", rows=32 * 196, C=384),
        # its gradient at the benchmark's shape
        dict(name="ln_bwd bf16 32768x1024", op="ln_bwd", dtype="bf16", rows=8 * 4096, C=1024),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "ln_fwd", "ln_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("ln_fwd", "ln_bwd"):
        C = rng.choice([192, 384, 768, 1024, rng.randint(33, 1100), 8 * rng.randint(5, 256)])
        return dict(op=op, dtype=dtype, rows=min(_log(rng, 1, 32768), (1 << 25) // C), C=C)
    H = rng.randint(1, 16)
    D = rng.choice([64, 64, 64, 128, 128, 32, rng.randint(9, 128)])
    if op == "step":
        B = _log(rng, 1, 256)
        return dict(op=op, dtype=dtype, B=B, H=H, D=D, pool=B + rng.randint(0, 40))
    T = _log(rng, 1, 16384)
    # the largest listed cases hold 8 * 4096 * 1024 values a tensor in bfloat16; float32 ones stay below
    most = (1 << 25 if op == "fwd" else 1 << 24) // (4 if dtype == "f32" else 1)
    B = max(1, min(_log(rng, 1, 64), most // (T * H * D)))
    T = max(1, min(T, most // (B * H * D)))
    case = dict(op=op, dtype=dtype, B=B, T=T, H=H, D=D, packed=rng.random() < 0.5, lens=rng.random() < 0.4, state=rng.random() < 0.5)
    return dict(case, want=rng.random() < 0.5) if op == "fwd" else case


def _lengths(case):
    """The sequences' lengths: fixed by the case, the longest of them T."""
    rng = random.Random(case["B"] * 1000003 + case["T"])
    n = [rng.randint(0, case["T"]) for _ in range(case["B"])]
    n[rng.randrange(case["B"])] = case["T"]
    return n


def _state_gradient(case):
    """Whether a loss also reaches the final state: sequences trained in pieces."""
    return case["state"]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    dtype = DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] in ("ln_fwd", "ln_bwd"):
        R, C = case["rows"], case["C"]
        # rows as a residual stream has them: a mean and a scale of their own
        x = normal(1, R, C) * (0.5 + 2.0 * torch.rand(1, R, 1, generator=g, device="cuda")) + normal(1, R, 1, std=0.5)
        st["x"] = x.to(dtype)
        st["gamma"], st["beta"] = 1.0 + normal(C, std=0.2), normal(C, std=0.2)
        if case["op"] == "ln_bwd":
            st["gy"] = normal(1, R, C, dtype=dtype)
            x = st["x"].double()  # the statistics that the forward pass kept
            st["mean"] = x.mean(-1).float()
            st["rstd"] = (x.var(-1, unbiased=False) + EPS).rsqrt().float()
        return st
    B, H, D = case["B"], case["H"], case["D"]
    # decays of the heads: half lives from about 2 to 400 tokens
    st["w"] = torch.exp(-0.7 - 5.6 * torch.rand(H, generator=g, device="cuda"))
    st["scale"] = D ** -0.5
    if case["op"] == "step":
        st["q"], st["k"], st["v"] = (normal(B, H * D, dtype=dtype) for _ in range(3))
        st["state"] = normal(case["pool"], H, D, D, std=4.0)
        st["slots"] = torch.randperm(case["pool"], generator=g, device="cuda")[:B].to(torch.int32)
        return st
    T = case["T"]
    if case["packed"]:
        st["q"], st["k"], st["v"] = normal(B, T, 3 * H * D, dtype=dtype).chunk(3, dim=-1)
    else:
        st["q"], st["k"], st["v"] = (normal(B, T, H * D, dtype=dtype) for _ in range(3))
    st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["lens"] else None
    st["state"] = normal(B, H, D, D, std=4.0) if case["state"] else None
    if case["op"] == "bwd":
        st["gy"] = normal(B, T, H * D, dtype=dtype)
        st["gstate"] = normal(B, H, D, D, std=4.0) if _state_gradient(case) else None
    return st


EPS = 1e-5


def run(st):
    case = st["case"]
    return (_own if own else _plain)[case["op"]](st, case)


# ---- the framework's calls -------------------------------------------------


def _own_fwd(st, case):
    import linear_complexity_vision_b200 as vk
    out, state = vk.decay_attn_fwd(st["q"], st["k"], st["v"], st["w"], case["H"], scale=st["scale"], state=st["state"],
                                   lengths=st["lengths"], want_state=case["want"])
    return {"out": out, "state": state} if case["want"] else {"out": out}


def _own_bwd(st, case):
    import linear_complexity_vision_b200 as vk
    gq, gk, gv, gs = vk.decay_attn_bwd(st["q"], st["k"], st["v"], st["w"], case["H"], st["gy"], scale=st["scale"],
                                       state=st["state"], gstate=st["gstate"], lengths=st["lengths"])
    return {"gq": gq, "gk": gk, "gv": gv, "gs": gs} if case["state"] else {"gq": gq, "gk": gk, "gv": gv}


def _own_step(st, case):
    import linear_complexity_vision_b200 as vk
    out = vk.decay_attn_step(st["q"], st["k"], st["v"], st["w"], case["H"], st["state"], slots=st["slots"], scale=st["scale"])
    return {"out": out, "state": st["state"]}


def _own_ln_fwd(st, case):
    import linear_complexity_vision_b200 as vk
    y, mean, rstd = vk.layer_norm_fwd(st["x"], st["gamma"], st["beta"], eps=EPS)
    return {"y": y, "mean": mean, "rstd": rstd}


def _own_ln_bwd(st, case):
    import linear_complexity_vision_b200 as vk
    gx, ggamma, gbeta = vk.layer_norm_bwd(st["x"], st["gamma"], st["mean"], st["rstd"], st["gy"])
    return {"gx": gx, "ggamma": ggamma, "gbeta": gbeta}


_own = {"fwd": _own_fwd, "bwd": _own_bwd, "step": _own_step, "ln_fwd": _own_ln_fwd, "ln_bwd": _own_ln_bwd}


# ---- the plain forms -------------------------------------------------------

CHUNK = 128


def _heads(x, st, T, pad):
    """(B, T, C) -> float32 (B, H, chunks, CHUNK, D), zero past the sequences' ends."""
    case = st["case"]
    x = x.float().view(case["B"], T, case["H"], case["D"])
    if st["lengths"] is not None:
        live = torch.arange(T, device="cuda")[None, :] < st["lengths"][:, None]
        x = torch.where(live[:, :, None, None], x, 0.0)
    x = torch.nn.functional.pad(x.transpose(1, 2), (0, 0, 0, pad))
    return x.reshape(case["B"], case["H"], -1, CHUNK, case["D"])


def _decay(w, n):
    """e^{-w n}, formed in 64 bits; 0 where n < 0."""
    n = n.double()
    return torch.where(n >= 0, torch.exp(-w.double() * n.clamp(min=0)), 0.0).float()


def _scan(q, k, v, w):
    """sum_{s <= t} e^{-w (t - s)} (q_t . k_s) v_s over chunks, all of them at once."""
    H, nc, D = q.shape[1], q.shape[2], q.shape[4]
    i = torch.arange(CHUNK, device="cuda")
    wh = w.view(H, 1, 1)
    inside = ((q @ k.transpose(-1, -2)) * _decay(wh, i[:, None] - i[None, :])[None, :, None]) @ v
    u = (k * _decay(w.view(H, 1), CHUNK - 1 - i)[None, :, None, :, None]).transpose(-1, -2) @ v  # each chunk's own sum at its end
    c = torch.arange(nc, device="cuda")
    across = _decay(wh, (c[:, None] - 1 - c[None, :]) * CHUNK)  # of chunk c' in the state before chunk c
    before = (across[None] @ u.flatten(3)).view_as(u)
    return inside + (q * _decay(w.view(H, 1), i + 1)[None, :, None, :, None]) @ before


def _tokens(x, T, dtype):
    """(B, H, chunks, CHUNK, D) -> (B, T, C), rounded once."""
    B, H, _, _, D = x.shape
    return x.reshape(B, H, -1, D)[:, :, :T].transpose(1, 2).reshape(B, T, H * D).to(dtype)


def _from_ends(st, T, pad):
    """Decays from the start state to each token, and from each token to the sequence's end; and over a whole sequence."""
    case, w = st["case"], st["w"].view(1, -1, 1)
    t = torch.arange(T + pad, device="cuda").view(1, 1, -1)
    n = torch.full((case["B"],), T, device="cuda") if st["lengths"] is None else st["lengths"].long()
    n = n.view(-1, 1, 1)
    shape = (case["B"], case["H"], -1, CHUNK, 1)
    since, until = _decay(w, (t + 1).expand(case["B"], -1, -1)), _decay(w, n - 1 - t)
    return since.reshape(shape), until.reshape(shape), _decay(w, n).unsqueeze(-1)


def _plain_fwd(st, case):
    T = case["T"]
    pad = -T % CHUNK
    q, k, v = (_heads(st[n], st, T, pad) for n in "qkv")
    since, until, over = _from_ends(st, T, pad)
    out = _scan(q, k, v, st["w"])
    if case["state"]:
        out = out + (q * since) @ st["state"].unsqueeze(2)
    got = {"out": _tokens(out * st["scale"], T, DTYPES[case["dtype"]])}
    if case["want"]:
        got["state"] = (k * until).flatten(2, 3).transpose(-1, -2) @ v.flatten(2, 3)
        if case["state"]:
            got["state"] = got["state"] + over * st["state"]
    return got


def _plain_bwd(st, case):
    T, s, dtype = case["T"], st["scale"], DTYPES[case["dtype"]]
    pad = -T % CHUNK
    q, k, v, g = (_heads(st[n], st, T, pad) for n in ("q", "k", "v", "gy"))
    since, until, over = _from_ends(st, T, pad)

    def back(a, b, c):  # the same sums over s >= t
        return _scan(a.flip(2, 3), b.flip(2, 3), c.flip(2, 3), st["w"]).flip(2, 3)

    gq, gk, gv = s * _scan(g, v, k, st["w"]), s * back(v, g, q), s * back(k, q, g)
    if case["state"]:
        s0, gs = st["state"].unsqueeze(2), st["gstate"].unsqueeze(2)
        gq = gq + s * (g * since) @ s0.transpose(-1, -2)
        gk = gk + (v * until) @ gs.transpose(-1, -2)
        gv = gv + (k * until) @ gs
    got = {"gq": _tokens(gq, T, dtype), "gk": _tokens(gk, T, dtype), "gv": _tokens(gv, T, dtype)}
    if case["state"]:
        got["gs"] = s * ((q * since).flatten(2, 3).transpose(-1, -2) @ g.flatten(2, 3)) + over * st["gstate"]
    return got


def _plain_step(st, case):
    B, H, D = case["B"], case["H"], case["D"]
    q, k, v = (st[n].float().view(B, H, 1, D) for n in "qkv")
    slots = st["slots"].long()
    s = st["state"][slots] * _decay(st["w"], torch.ones_like(st["w"])).view(1, H, 1, 1) + k.transpose(-1, -2) * v
    st["state"][slots] = s
    return {"out": (st["scale"] * (q @ s)).reshape(B, H * D).to(DTYPES[case["dtype"]]), "state": st["state"]}


def _plain_ln_fwd(st, case):
    x = st["x"].float()
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + EPS).rsqrt()
    y = (x - mean) * rstd * st["gamma"] + st["beta"]
    return {"y": y.to(st["x"].dtype), "mean": mean.squeeze(-1), "rstd": rstd.squeeze(-1)}


def _plain_ln_bwd(st, case):
    g, rstd = st["gy"].float(), st["rstd"].unsqueeze(-1)
    xh = (st["x"].float() - st["mean"].unsqueeze(-1)) * rstd
    d = g * st["gamma"]
    gx = rstd * (d - d.mean(-1, keepdim=True) - xh * (d * xh).mean(-1, keepdim=True))
    return {"gx": gx.to(st["x"].dtype), "ggamma": (g * xh).sum((0, 1)), "gbeta": g.sum((0, 1))}


_plain = {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd}


# ---- in 64 bits, token by token -------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("ln_fwd", "ln_bwd"):
        x, gamma = st["x"].double(), st["gamma"].double()
        if case["op"] == "ln_fwd":
            var, mean = torch.var_mean(x, -1, unbiased=False, keepdim=True)
            std = torch.sqrt(var + EPS)
            return {"y": gamma * ((x - mean) / std) + st["beta"].double(), "mean": mean.squeeze(-1), "rstd": 1.0 / std.squeeze(-1)}
        g, rstd = st["gy"].double(), st["rstd"].double().unsqueeze(-1)
        xh = (x - st["mean"].double().unsqueeze(-1)) * rstd
        gh = gamma * g
        a = torch.einsum("brc->br", gh).unsqueeze(-1) / case["C"]
        b = torch.einsum("brc,brc->br", gh, xh).unsqueeze(-1) / case["C"]
        return {"gx": (gh - a - b * xh) * rstd, "ggamma": torch.einsum("brc,brc->c", g, xh), "gbeta": torch.einsum("brc->c", g)}
    B, H, D = case["B"], case["H"], case["D"]
    lam = torch.exp(-st["w"].double()).view(1, H, 1, 1)
    if case["op"] == "step":
        q, k, v = (st[n].double().view(B, H, D) for n in "qkv")
        pool = st["state"].double()
        out = torch.empty_like(q)
        for b, slot in enumerate(st["slots"].tolist()):
            pool[slot] = lam[0] * pool[slot] + torch.einsum("hi,hj->hij", k[b], v[b])
            out[b] = st["scale"] * torch.einsum("hi,hij->hj", q[b], pool[slot])
        return {"out": out.view(B, H * D), "state": pool}
    T = case["T"]
    live = torch.ones(T, B, 1, 1, 1, dtype=torch.bool, device="cuda")
    if case["lens"]:
        live = (torch.arange(T, device="cuda")[:, None] < st["lengths"][None, :]).view(T, B, 1, 1, 1)
    # the tokens past a sequence's end are zeros that its states pass by
    q, k, v = (torch.where(live[:, :, 0], st[n].transpose(0, 1).double().reshape(T, B, H, D), 0.0) for n in "qkv")
    S = st["state"].double() if case["state"] else torch.zeros(B, H, D, D, dtype=torch.float64, device="cuda")
    if case["op"] == "fwd":
        out = torch.zeros(B, T, H, D, dtype=torch.float64, device="cuda")
        for t in range(T):
            S = torch.where(live[t], torch.baddbmm((lam * S).flatten(0, 1), k[t].reshape(-1, D, 1), v[t].reshape(-1, 1, D)).view_as(S), S)
            out[:, t] = st["scale"] * (q[t].unsqueeze(-2) @ S).squeeze(-2)
        got = {"out": out.view(B, T, H * D)}
        return dict(got, state=S) if case["want"] else got
    g = torch.where(live[:, :, 0], st["gy"].transpose(0, 1).double().reshape(T, B, H, D), 0.0)
    gq, gk, gv = (torch.zeros(B, T, H, D, dtype=torch.float64, device="cuda") for _ in range(3))
    for t in range(T):
        S = torch.where(live[t], torch.baddbmm((lam * S).flatten(0, 1), k[t].reshape(-1, D, 1), v[t].reshape(-1, 1, D)).view_as(S), S)
        gq[:, t] = st["scale"] * (S @ g[t].unsqueeze(-1)).squeeze(-1)
    G = st["gstate"].double() if case["state"] else torch.zeros(B, H, D, D, dtype=torch.float64, device="cuda")
    for t in range(T - 1, -1, -1):  # G: the loss's gradient with respect to S_t
        G = torch.baddbmm(G.flatten(0, 1), st["scale"] * q[t].reshape(-1, D, 1), g[t].reshape(-1, 1, D)).view_as(G)
        gk[:, t] = (G @ v[t].unsqueeze(-1)).squeeze(-1)
        gv[:, t] = (k[t].unsqueeze(-2) @ G).squeeze(-2)
        G = torch.where(live[t], lam * G, G)
    got = {"gq": gq.view(B, T, H * D), "gk": gk.view(B, T, H * D), "gv": gv.view(B, T, H * D)}
    return dict(got, gs=G) if case["state"] else got


def work(case):
    """Bytes: each input read once, each output written once; the tokens past a sequence's end are only written.
    Operations: those of the recurrence, a product of the token with the state and one that updates it."""
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "ln_fwd":
        n = case["rows"] * case["C"]
        return {"bytes": 2 * n * es + 8 * case["rows"] + 8 * case["C"], "flops": 8 * n}
    if case["op"] == "ln_bwd":
        n = case["rows"] * case["C"]
        return {"bytes": 3 * n * es + 8 * case["rows"] + 12 * case["C"], "flops": 14 * n}
    B, H, D = case["B"], case["H"], case["D"]
    if case["op"] == "step":
        return {"bytes": B * (2 * H * D * D * 4 + 4 * H * D * es + 4) + 4 * H, "flops": B * H * 5 * D * D}
    tokens, live = B * case["T"], sum(_lengths(case)) if case["lens"] else B * case["T"]
    states = B * H * D * D * 4
    if case["op"] == "fwd":
        return {"bytes": (3 * live + tokens) * H * D * es + states * (case["state"] + case["want"]), "flops": 4 * live * H * D * D}
    return {"bytes": (4 * live + 3 * tokens) * H * D * es + 3 * states * case["state"], "flops": 10 * live * H * D * D}
