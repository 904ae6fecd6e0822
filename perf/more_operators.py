"""The gated delta rule and the norm of its keys and queries, as a user calls them, and their plain forms.

  forward        the gated delta rule over sequences (dense or packed), by chunks
  backward       its gradients, the states recomputed
  step           one token per sequence, the fp32 state updated in place (decoding)
  norm           keys B and queries C normalised per head, rotated by their positions in the same pass
  norm_backward  its gradients

``own`` False: elementary torch operations in 32 bits (angles and sums over tokens in 64), rounded
once at the end. ``own`` True: the framework's operators.
"""
import math
import random

import torch

own = False

CHUNK = 64       # tokens that the plain form takes at once
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # prefill or a training pass of the 2.7B-shaped layer (8 sequences of 2048 tokens)
        dict(name="forward 8 x 2048", op="forward", batch=8, seqlen=2048, num_seqs=0, max_len=0,
             len_seed=0, heads=80, headdim=64, dstate=128, groups=1, dtype="bf16", state=False),
        # prefill of one long prompt continued from a state: few heads, many chunks in a row
        dict(name="forward 1 x 16384", op="forward", batch=1, seqlen=16384, num_seqs=0, max_len=0,
             len_seed=0, heads=32, headdim=128, dstate=128, groups=16, dtype="bf16", state=True),
        # packed prompts of 16 to 1536 tokens, the small layer
        dict(name="forward packed", op="forward", batch=1, seqlen=0, num_seqs=48, max_len=1536,
             len_seed=7, heads=24, headdim=64, dstate=128, groups=1, dtype="bf16", state=False),
        # a short fp32 segment continued from a state, odd length, three groups
        dict(name="forward fp32", op="forward", batch=3, seqlen=257, num_seqs=0, max_len=0,
             len_seed=0, heads=12, headdim=64, dstate=64, groups=3, dtype="fp32", state=True),
        # training, two heads to a key, the states long as wide
        dict(name="backward 4 x 2048", op="backward", batch=4, seqlen=2048, num_seqs=0, max_len=0,
             len_seed=0, heads=32, headdim=128, dstate=128, groups=16, dtype="bf16", state=False),
        # training on packed sequences in fp32, from states, odd lengths
        dict(name="backward packed fp32", op="backward", batch=1, seqlen=0, num_seqs=6,
             max_len=500, len_seed=3, heads=8, headdim=64, dstate=64, groups=2, dtype="fp32",
             state=True),
        # decoding one sequence, where latency counts
        dict(name="step, 1 sequence", op="step", batch=1, heads=24, headdim=64, dstate=128,
             groups=1, dtype="bf16"),
        # decoding 256 sequences of the 2.7B-shaped layer
        dict(name="step, 256 sequences", op="step", batch=256, heads=80, headdim=64, dstate=128,
             groups=1, dtype="bf16"),
        # decoding 16 sequences: keys and queries of 16 heads of one token each, far positions
        dict(name="norm, 16 tokens", op="norm", tokens=16, b_heads=16, c_heads=16, dim=128,
             dtype="bf16", rotary=64, interleaved=False, unit=False, start=100000, pad=0),
        # a training or prefill pass: unit keys and queries, slices of wider rows, no rotation
        dict(name="norm, 16384 tokens", op="norm", tokens=16384, b_heads=16, c_heads=16, dim=128,
             dtype="bf16", rotary=0, interleaved=False, unit=True, start=0, pad=4096),
        # its gradients, fully rotated, queries with more heads than keys
        dict(name="norm backward", op="norm_backward", tokens=16384, b_heads=8, c_heads=32, dim=128,
             dtype="bf16", rotary=128, interleaved=False, unit=False, start=0, pad=0),
        # one wide group each, fp32, pairs side by side, an odd count
        dict(name="norm backward fp32", op="norm_backward", tokens=4099, b_heads=1, c_heads=1,
             dim=256, dtype="fp32", rotary=128, interleaved=True, unit=False, start=0, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above: 1 to 4096 tokens a sequence, 1 to 64 sequences, 1 to 80
    heads in any grouping, every head size, 1 to 16384 tokens to normalise, both types."""
    op = rng.choice(["forward", "forward", "forward", "backward", "backward", "step", "norm",
                     "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("norm", "norm_backward"):
        dim = 16 * _log(rng, 1, 16)
        b_heads = _log(rng, 1, 32)
        c_heads = rng.choice([b_heads, _log(rng, 1, 32)])
        tokens = _log(rng, 1, min(16384, (1 << 26) // (dim * (b_heads + c_heads))))
        return dict(op=op, tokens=tokens, b_heads=b_heads, c_heads=c_heads, dim=dim, dtype=dtype,
                    rotary=rng.choice([0, dim, 16 * rng.randint(0, dim // 16)]),
                    interleaved=rng.random() < 0.5, unit=rng.random() < 0.5,
                    start=rng.choice([0, _log(rng, 1, 1 << 20)]),
                    pad=rng.choice([0, 0, 8 * rng.randint(1, 600)]))
    groups = _log(rng, 1, 16)
    heads = groups * _log(rng, 1, max(1, 80 // groups))
    headdim = rng.choice([16, 32, 64, 64, 128, 128])
    dstate = 16 * _log(rng, 1, 16)
    c = dict(op=op, heads=heads, headdim=headdim, dstate=dstate, groups=groups, dtype=dtype)
    if op == "step":
        c["batch"] = _log(rng, 1, max(1, min(256, (1 << 27) // (heads * headdim * dstate))))
        return c
    most = (1 << 28) // (heads * (headdim + dstate)) // (4 if op == "backward" else 1)
    c.update(batch=1, seqlen=0, num_seqs=0, max_len=0, len_seed=0, state=rng.random() < 0.5)
    if rng.random() < 0.5:
        c["batch"] = _log(rng, 1, 8)
        c["seqlen"] = _log(rng, 1, min(4096, max(2, most // c["batch"])))
    else:
        c["num_seqs"] = _log(rng, 1, 64)
        c["max_len"] = _log(rng, 2, min(2048, max(3, most // c["num_seqs"])))
        c["len_seed"] = rng.randrange(1 << 20)
    return c


def _lengths(case):
    """The sequences' lengths; packed ones spread evenly from 16 (or 0, where that is short)."""
    if not case["num_seqs"]:
        return [case["seqlen"]] * case["batch"]
    r = random.Random(case["len_seed"])
    low = 16 if case["max_len"] > 64 else 0
    lens = [r.randint(low, case["max_len"]) for _ in range(case["num_seqs"])]
    lens[-1] = max(lens[-1], 1)
    return lens


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("norm", "norm_backward"):
        n = case["tokens"] * (case["b_heads"] + case["c_heads"]) * case["dim"]
        extra = 8 * case["dim"] + (4 * case["tokens"] + 2 * case["rotary"] if case["rotary"] else 0)
        if op == "norm":
            return {"bytes": 2 * n * es + extra, "flops": 8 * n}
        return {"bytes": 3 * n * es + extra + 8 * case["dim"], "flops": 18 * n}
    H, P, N, G = case["heads"], case["headdim"], case["dstate"], case["groups"]
    if op == "step":
        b = case["batch"]
        return {"bytes": b * (8 * H * P * N + es * (2 * H * P + 2 * H + 2 * G * N)),
                "flops": 7 * b * H * P * N}
    lens = _lengths(case)
    T, S = sum(lens), len(lens)
    token = es * (H * P + 2 * H + 2 * G * N)
    given = 4 * S * H * P * N if case["state"] else 0
    if op == "forward":
        return {"bytes": T * (token + es * H * P) + given + 4 * S * H * P * N,
                "flops": 7 * T * H * P * N}
    return {"bytes": T * (2 * token + es * H * P) + 3 * given, "flops": 20 * T * H * P * N}


# ---- inputs ------------------------------------------------------------------


def _inputs(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    s = dict(case=case)
    if op in ("norm", "norm_backward"):
        T, N = case["tokens"], case["dim"]
        for name, heads in (("B", case["b_heads"]), ("C", case["c_heads"])):
            # activations of channels of different sizes, a few rows far larger; both lie in
            # rows with other channels between them
            v = rand(T, heads * N) * torch.exp(0.5 * rand(1, heads * N)) * torch.exp(0.5 * rand(T, 1))
            wide = torch.zeros(T, heads * N + case["pad"], device="cuda", dtype=dt)
            wide[:, :heads * N] = v.to(dt)
            s[name] = wide[:, :heads * N].unflatten(1, (heads, N))
            s[name + "_weight"] = 1 + 0.1 * rand(N)
            if op == "norm_backward":
                s["d" + name] = (0.1 * rand(T, heads, N)).to(dt)
        s["positions"] = s["freqs"] = None
        if case["rotary"]:
            s["positions"] = torch.arange(T, device="cuda", dtype=torch.int32) + case["start"]
            i = torch.arange(case["rotary"] // 2, device="cuda", dtype=torch.float64)
            s["freqs"] = (10000.0 ** (-2 * i / case["rotary"])).float()
        return s
    H, P, N, G = case["heads"], case["headdim"], case["dstate"], case["groups"]
    lead = (case["batch"],) if op == "step" else \
        (1, sum(_lengths(case))) if case["num_seqs"] else (case["batch"], case["seqlen"])
    S = lead[0] if op == "step" else len(_lengths(case))
    s["x"] = rand(*lead, H, P).to(dt)
    # steps of 0.001 to 0.1 and rates of 1 to 16, as the layer has them; writes of any strength
    step = torch.exp(rand(*lead, H).sigmoid() * math.log(100.0) + math.log(0.001))
    rate = 1 + 15 * torch.rand(H, device="cuda", generator=g)
    s["g"] = (-step * rate).to(dt)
    s["beta"] = torch.sigmoid(rand(*lead, H)).to(dt)
    # unit keys that have a part in common, and queries
    for name in ("B", "C"):
        v = rand(*lead, G, N) + 0.5 * rand(G, N)
        size = torch.sqrt((v * v).sum(-1, keepdim=True)) if name == "B" else N ** 0.5
        s[name] = (v / size).to(dt)
    s["state"] = 0.3 * rand(S, H, P, N) if op == "step" or case["state"] else None
    s["cu"] = None
    if op != "step" and case["num_seqs"]:
        ends = torch.tensor(_lengths(case), device="cuda").cumsum(0)
        s["cu"] = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    if op == "backward":
        s["dy"] = (0.1 * rand(*lead, H, P)).to(dt)
        s["dstate"] = 0.1 * rand(S, H, P, N) if case["state"] else None
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ---- the framework's operators -------------------------------------------------


def _run_own(s):
    import mamba_ssd_sequence_fwd_amd as ssd
    c = s["case"]
    op = c["op"]
    if op == "step":
        return [ssd.delta_step(s["x"], s["g"], s["beta"], s["B"], s["C"], s["state"]), s["state"]]
    if op == "forward":
        return list(ssd.delta_forward(s["x"], s["g"], s["beta"], s["B"], s["C"], s["state"],
                                      s["cu"], check_cu_seqlens=False))
    if op == "backward":
        d = ssd.delta_backward(s["x"], s["g"], s["beta"], s["B"], s["C"], s["state"], s["dy"],
                               s["dstate"], s["cu"], check_cu_seqlens=False)
        return [d[k] for k in ("dx", "dg", "dbeta", "dB", "dC")] + \
            ([d["dinitial_state"]] if c["state"] else [])
    kw = dict(eps=EPS, unit=c["unit"], interleaved=c["interleaved"])
    if op == "norm":
        return list(ssd.bc_norm(s["B"], s["C"], s["B_weight"], s["C_weight"], s["positions"],
                                s["freqs"], **kw))
    d = ssd.bc_norm_backward(s["dB"], s["dC"], s["B"], s["C"], s["B_weight"], s["C_weight"],
                             s["positions"], s["freqs"], **kw)
    return [d[k] for k in ("dB", "dC", "dB_weight", "dC_weight")]


# ---- the plain forms: keys and queries -------------------------------------------


def _turn(v, cos, sin, interleaved, back=False):
    """The first 2 * cos.shape[-1] channels of v (tokens, heads, N) turned by pairs."""
    r = cos.shape[-1]
    cos, sin = cos[:, None], (-sin if back else sin)[:, None]
    rest = v[..., 2 * r:]
    if interleaved:
        a, b = v[..., 0:2 * r:2], v[..., 1:2 * r:2]
        return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest], -1)
    a, b = v[..., :r], v[..., r:2 * r]
    return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)


def _plain_norm(s, backward):
    c = s["case"]
    cos = sin = None
    if c["rotary"]:
        angle = s["positions"].double()[:, None] * s["freqs"].double()
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    outs, sums = [], []
    for name in ("B", "C"):
        x, w = s[name].float(), s[name + "_weight"]
        n = 1 if c["unit"] else c["dim"]
        r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / n + EPS)
        if not backward:
            v = x * r * w
            outs.append((v if cos is None else _turn(v, cos, sin, c["interleaved"])).to(s[name].dtype))
            continue
        d = s["d" + name].float()
        if cos is not None:
            d = _turn(d, cos, sin, c["interleaved"], back=True)
        h, dh = x * r, d * w
        sums.append((d * h).sum((0, 1), dtype=torch.float64).float())
        outs.append((r * (dh - h * ((dh * h).sum(-1, keepdim=True) / n))).to(s[name].dtype))
    return outs + sums


# ---- the plain forms: the delta rule by chunks --------------------------------------


def _rows(s):
    """(place of each token in (sequences, padded length), sequences, padded length)."""
    lens = _lengths(s["case"])
    longest = -(-max(max(lens), 1) // CHUNK) * CHUNK
    if s["cu"] is None:
        tok = torch.arange(len(lens) * lens[0], device="cuda")
        return tok // max(lens[0], 1) * longest + tok % max(lens[0], 1), len(lens), longest
    cu = s["cu"].long()
    tok = torch.arange(sum(lens), device="cuda")
    seq = torch.searchsorted(cu, tok, right=True) - 1
    return seq * longest + tok - cu[seq], len(lens), longest


def _chunks(t, at, S, longest, heads):
    """(S, heads, chunks, CHUNK, channels) of t (batch, L, groups[, channels]), 0 where no token
    is: such a row neither decays nor writes."""
    t = t.reshape(at.shape[0], t.shape[2], -1).float()
    p = t.new_zeros(S * longest, *t.shape[1:])
    p[at] = t
    p = p.view(S, longest // CHUNK, CHUNK, *t.shape[1:]).permute(0, 3, 1, 2, 4)
    r = heads // t.shape[1]
    return p.repeat_interleave(r, 1) if r > 1 else p.contiguous()


def _tokens(p, at, groups, like):
    """_chunks back: (batch, L, groups[, channels]), the heads of a group summed."""
    S, H, nc, c, n = p.shape
    p = p.view(S, groups, H // groups, nc, c, n).sum(2)
    p = p.permute(0, 2, 3, 1, 4).reshape(S * nc * c, groups * n)[at]
    return p.reshape(like.shape).to(like.dtype)


def _parts(s):
    c = s["case"]
    at, S, longest = _rows(s)
    K, Q, V, g, beta = (_chunks(s[k], at, S, longest, c["heads"]) for k in ("B", "C", "x", "g", "beta"))
    gam = torch.cumsum(g, 3)
    low = torch.ones(CHUNK, CHUNK, device="cuda", dtype=torch.bool).tril()
    D = torch.where(low, gam - gam.transpose(3, 4), -math.inf).exp()
    KD = (K @ K.transpose(3, 4)) * D
    KD = KD.tril(-1)
    M = (Q @ K.transpose(3, 4)) * D
    Lm = beta * KD
    T = torch.zeros_like(Lm)
    T[..., 0, 0] = 1
    for i in range(1, CHUNK):              # (I + L)^-1 row by row
        T[..., i, :i] = -(Lm[..., i:i + 1, :i] @ T[..., :i, :i])[..., 0, :]
        T[..., i, i] = 1
    end = gam[..., -1:, :]
    return dict(at=at, S=S, K=K, Q=Q, V=V, beta=beta, D=D, KD=KD, M=M, Lm=Lm, T=T,
                fall=gam.exp(), left=(end - gam).exp(), end=end.exp())


def _first_state(s, p):
    c = s["case"]
    if s["state"] is None:
        return p["K"].new_zeros(p["S"], c["heads"], c["dstate"], c["headdim"])
    return s["state"].transpose(2, 3).contiguous()


def _plain_forward(s):
    p = _parts(s)
    w = p["T"] @ (p["beta"] * p["fall"] * p["K"])
    u = p["T"] @ (p["beta"] * p["V"])
    kl, qf = (p["left"] * p["K"]).transpose(3, 4), p["fall"] * p["Q"]
    st = _first_state(s, p)
    y = torch.empty_like(p["V"])
    for k in range(y.shape[2]):
        uk = u[:, :, k] - w[:, :, k] @ st
        y[:, :, k] = qf[:, :, k] @ st + p["M"][:, :, k] @ uk
        st = p["end"][:, :, k] * st + kl[:, :, k] @ uk
    return [_tokens(y, p["at"], s["case"]["heads"], s["x"]), st.transpose(2, 3).contiguous()]


def _plain_backward(s):
    c = s["case"]
    p = _parts(s)
    K, Q, V, T, M, D, beta = (p[k] for k in ("K", "Q", "V", "T", "M", "D", "beta"))
    fall, left, end = p["fall"], p["left"], p["end"]
    dY = _chunks(s["dy"], p["at"], p["S"], p["D"].shape[2] * CHUNK, c["heads"])
    st = _first_state(s, p)
    nc = V.shape[2]
    S0 = V.new_empty(p["S"], c["heads"], nc, c["dstate"], c["headdim"])
    U = torch.empty_like(V)
    w, u, kl = T @ (beta * fall * K), T @ (beta * V), (left * K).transpose(3, 4)
    for k in range(nc):
        S0[:, :, k] = st
        U[:, :, k] = u[:, :, k] - w[:, :, k] @ st
        st = end[:, :, k] * st + kl[:, :, k] @ U[:, :, k]
    dS1, dR = torch.empty_like(S0), torch.empty_like(V)
    du, lk = M.transpose(3, 4) @ dY, left * K
    qt, kt, Tt = (fall * Q).transpose(3, 4) @ dY, (beta * fall * K).transpose(3, 4), T.transpose(3, 4)
    ds = torch.zeros_like(st) if s["dstate"] is None else s["dstate"].transpose(2, 3).contiguous()
    for k in range(nc - 1, -1, -1):
        dS1[:, :, k] = ds
        dR[:, :, k] = Tt[:, :, k] @ (du[:, :, k] + lk[:, :, k] @ ds)
        ds = end[:, :, k] * ds + qt[:, :, k] - kt[:, :, k] @ dR[:, :, k]
    dM = (dY @ U.transpose(3, 4)).tril()
    dL = -(dR @ U.transpose(3, 4)).tril(-1)
    S0t = S0.transpose(3, 4)
    dq, dk = fall * (dY @ S0t), -fall * (dR @ S0t)       # dk still without beta
    dkl = left * (U @ dS1.transpose(3, 4))
    dbeta = (dR * V).sum(-1, keepdim=True) + (dk * K).sum(-1, keepdim=True) + \
        (dL * p["KD"]).sum(-1, keepdim=True)
    # each decay's log: what lies at or behind it against what lies before it
    a = (dq * Q).sum(-1, keepdim=True) + beta * (dk * K).sum(-1, keepdim=True)
    b = (dkl * K).sum(-1, keepdim=True)
    W = dM * M + dL * p["Lm"]
    over = torch.flip(torch.cumsum(torch.flip(W, [3]), 3), [3])      # sums over rows i >= t
    dg = torch.flip(torch.cumsum(torch.flip(a, [3]), 3), [3]) + torch.cumsum(b, 3) - b \
        + over.tril(-1).sum(-1, keepdim=True) + end * (S0 * dS1).sum((3, 4), keepdim=True)
    dMd, dLd = dM * D, dL * beta * D
    dQ = dq + dMd @ K
    dK = beta * dk + dkl + dMd.transpose(3, 4) @ Q + dLd @ K + dLd.transpose(3, 4) @ K
    outs = [_tokens(t, p["at"], n, s[k]) for t, n, k in (
        (beta * dR, c["heads"], "x"), (dg, c["heads"], "g"), (dbeta, c["heads"], "beta"),
        (dK, c["groups"], "B"), (dQ, c["groups"], "C"))]
    return outs + ([ds.transpose(2, 3).contiguous()] if c["state"] else [])


def _plain_step(s):
    c = s["case"]
    r = c["heads"] // c["groups"]
    K, Q = (s[k].float().repeat_interleave(r, 1)[..., None] for k in ("B", "C"))
    st = s["state"]
    st *= s["g"].float().exp()[..., None, None]
    e = s["beta"].float()[..., None, None] * (s["x"].float()[..., None] - st @ K)
    st += e * K.transpose(2, 3)
    return [(st @ Q)[..., 0].to(s["x"].dtype), st]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "forward":
        return _plain_forward(state)
    if op == "backward":
        return _plain_backward(state)
    if op == "step":
        return _plain_step(state)
    return _plain_norm(state, op == "norm_backward")


# ---- from the definition, in 64 bits: token by token ---------------------------------


def _exact_norm(s, backward):
    c = s["case"]
    outs, sums = [], []
    for name in ("B", "C"):
        x, w = s[name].double(), s[name + "_weight"].double()
        x.requires_grad_(backward)
        w.requires_grad_(backward)
        size = x.pow(2).sum(-1, keepdim=True) if c["unit"] else x.pow(2).mean(-1, keepdim=True)
        v = x * (size + EPS) ** -0.5 * w
        half = c["rotary"] // 2
        if half:
            turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64),
                               torch.outer(s["positions"].double(), s["freqs"].double()))
            z = v[..., :2 * half]
            z = z.unflatten(-1, (half, 2)) if c["interleaved"] else \
                z.unflatten(-1, (2, half)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn[:, None])
            z = z if c["interleaved"] else z.transpose(-1, -2)
            v = torch.cat([z.flatten(-2), v[..., 2 * half:]], -1)
        if backward:
            dx, dw = torch.autograd.grad(v, (x, w), s["d" + name].double())
            outs.append(dx)
            sums.append(dw)
        else:
            outs.append(v)
    return outs + sums


def _padded(t, case, heads):
    """(L, sequences, heads, channels) in 64 bits, zeros behind a sequence's last token."""
    lens = _lengths(case)
    if not case["num_seqs"]:
        p = t.double().transpose(0, 1)
    else:
        p = torch.zeros(max(lens), len(lens), *t.shape[2:], device="cuda", dtype=torch.float64)
        at = 0
        for k, n in enumerate(lens):
            p[:n, k] = t[0, at:at + n].double()
            at += n
    p = p.reshape(*p.shape[:3], -1)
    return p.repeat_interleave(heads // p.shape[2], 2)


def _unpadded(rows, case, groups, like):
    p = torch.stack(rows) if isinstance(rows, list) else rows              # (L, S, H, n)
    p = p.unflatten(2, (groups, -1)).sum(3)
    if not case["num_seqs"]:
        return p.transpose(0, 1).reshape(like.shape)
    return torch.cat([p[:n, k] for k, n in enumerate(_lengths(case))]).reshape(like.shape)


def _advance(h, k, v, a, b):
    """One token: (decayed state, what it lacks of v, new state)."""
    d = h * a[..., None]
    e = v - (d @ k[..., None])[..., 0]
    return d, e, d + (b * e)[..., None] * k[:, :, None]


def _exact_delta(s):
    c = s["case"]
    H = c["heads"]
    K, Q, V, g, beta = (_padded(s[k], c, H) for k in ("B", "C", "x", "g", "beta"))
    a = g.exp()
    L, S = K.shape[:2]
    h = K.new_zeros(S, H, c["headdim"], c["dstate"]) if s["state"] is None else s["state"].double()
    part = max(1, min(256, int(2e10) // max(1, h.numel() * 8)))
    kept, y = [], []
    for t in range(L):
        if t % part == 0:
            kept.append(h)
        h = _advance(h, K[t], V[t], a[t], beta[t])[2]
        if c["op"] == "forward":
            y.append((h @ Q[t][..., None])[..., 0])
    if c["op"] == "forward":
        return [_unpadded(y, c, H, s["x"]), h]
    dY = _padded(s["dy"], c, H)
    G = torch.zeros_like(h) if s["dstate"] is None else s["dstate"].double()
    dK, dQ, dV, dg, db = (torch.zeros_like(t) for t in (K, Q, V, g, beta))
    for first in range((L - 1) // part * part, -1, -part):
        h = kept.pop()
        seen = []
        for t in range(first, min(L, first + part)):
            seen.append(_advance(h, K[t], V[t], a[t], beta[t]))
            h = seen[-1][2]
        for t in range(min(L, first + part) - 1, first - 1, -1):
            d, e, h = seen.pop()
            G = G + dY[t][..., None] * Q[t][:, :, None]
            Gk = (G @ K[t][..., None])[..., 0]
            dQ[t] = (dY[t][:, :, None] @ h)[:, :, 0]
            db[t] = (Gk * e).sum(-1, keepdim=True)
            dV[t] = beta[t] * Gk
            dK[t] = beta[t] * (e[:, :, None] @ G)[:, :, 0] - (dV[t][:, :, None] @ d)[:, :, 0]
            G = G - dV[t][..., None] * K[t][:, :, None]
            dg[t] = (G * d).sum((2, 3))[..., None]
            G = G * a[t][..., None]
    outs = [_unpadded(t, c, n, s[k]) for t, n, k in (
        (dV, H, "x"), (dg, H, "g"), (db, H, "beta"), (dK, c["groups"], "B"), (dQ, c["groups"], "C"))]
    return outs + ([G] if c["state"] else [])


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("norm", "norm_backward"):
        return _exact_norm(s, case["op"] == "norm_backward")
    if case["op"] != "step":
        return _exact_delta(s)
    one = dict(case, op="forward", seqlen=1, num_seqs=0, max_len=0, len_seed=0, state=True)
    s = dict(s, case=one, **{k: s[k][:, None] for k in ("x", "g", "beta", "B", "C")})
    y, h = _exact_delta(s)
    return [y[:, 0], h]
