"""The operators around the SSD layer, as a user calls them, and their plain forms.

  norm           group norm with SiLU (the gate behind the layer), channels last
  norm_backward  its gradients, from the stored inputs or from 8-bit checkpoints of them
  conv_backward  the gradients of the convolution front, from its input or an 8-bit checkpoint of it
  conv_save      the front, keeping its input in 8 bits on the way
  conv_load      the front recomputed from the 8-bit checkpoint (what the SSD backward pass reads)
  norm_save      the norm, keeping both of its inputs in 8 bits on the way
  save           an 8-bit checkpoint of any tensor, and its values again

``own`` False: elementary torch operations in 32 bits (sums over tokens in 64), rounded once at
the end. ``own`` True: the framework's operators.
"""
import math
import random

import torch

own = False

BLOCK = 32       # channels of one row that share a scale
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # decoding: the gate behind the 2.7B-shaped layer for one token, where latency counts
        dict(name="norm, 1 token", op="norm", tokens=1, channels=5120, groups=1, dtype="bf16",
             gate="first", center=False, bias=False, pad=5456),
        # a training or prefill pass of the 2.7B-shaped layer (8 sequences of 2048 tokens); z is a
        # column slice of the input projection's rows (z, xBC, dt)
        dict(name="norm, 16384 tokens", op="norm", tokens=16384, channels=5120, groups=1,
             dtype="bf16", gate="first", center=False, bias=False, pad=5456),
        # one group per head, mean taken off, affine, gate behind the norm, fp32, an odd count
        dict(name="norm per head fp32", op="norm", tokens=4099, channels=1536, groups=24,
             dtype="fp32", gate="last", center=True, bias=True, pad=0),
        # training, 2.7B-shaped layer, inputs stored as they are
        dict(name="norm backward", op="norm_backward", tokens=16384, channels=5120, groups=1,
             dtype="bf16", gate="first", center=False, bias=False, pad=5456, ckpt=False),
        # training, long sequences (2 of 16384 tokens), 8 groups, inputs from 8-bit checkpoints
        dict(name="norm backward 8-bit", op="norm_backward", tokens=32768, channels=4096, groups=8,
             dtype="bf16", gate="first", center=False, bias=False, pad=0, ckpt=True),
        # the classical form: no z, the activation behind an affine group norm; ragged, small
        dict(name="norm backward no gate", op="norm_backward", tokens=1023, channels=1280, groups=4,
             dtype="fp32", gate="none", center=True, bias=True, pad=0, ckpt=False),
        # training on 64 packed sequences of 16 to 4096 tokens: the largest pass
        dict(name="conv backward packed", op="conv_backward", batch=1, seqlen=0, num_seqs=64,
             max_len=4096, len_seed=4, x_dim=5120, bc_dim=128, width=4, dtype="bf16",
             history=False, ckpt=False),
        # training, the 2.7B-shaped front, its input from the 8-bit checkpoint
        dict(name="conv backward 8-bit", op="conv_backward", batch=8, seqlen=2048, num_seqs=0,
             max_len=0, len_seed=0, x_dim=5120, bc_dim=128, width=4, dtype="bf16", history=False,
             ckpt=True),
        # a short fp32 segment continued from a history, three taps, odd length
        dict(name="conv backward fp32", op="conv_backward", batch=3, seqlen=257, num_seqs=0,
             max_len=0, len_seed=0, x_dim=768, bc_dim=64, width=3, dtype="fp32", history=True,
             ckpt=False),
        # training forward: the 2.7B-shaped front, its input kept in 8 bits
        dict(name="conv save", op="conv_save", batch=8, seqlen=2048, num_seqs=0, max_len=0,
             len_seed=0, x_dim=5120, bc_dim=128, width=4, dtype="bf16", history=False),
        # the small layer's front recomputed for its backward pass
        dict(name="conv from 8-bit", op="conv_load", batch=4, seqlen=2048, num_seqs=0, max_len=0,
             len_seed=0, x_dim=1536, bc_dim=128, width=4, dtype="bf16", history=False),
        # training forward with 8 groups, both inputs of the norm kept in 8 bits
        dict(name="norm save", op="norm_save", tokens=32768, channels=4096, groups=8, dtype="bf16",
             gate="first", center=False, bias=False, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above: 1 to 32768 tokens, 8 to 8192 channels (multiples of 8),
    groups from 8 channels to the whole row, both types, every form."""
    op = rng.choice(["norm", "norm", "norm_backward", "norm_backward", "conv_backward",
                     "conv_backward", "conv_save", "conv_load", "norm_save", "save"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("norm", "norm_backward", "norm_save", "save"):
        gs = 8 * _log(rng, 1, 1024)
        groups = _log(rng, 1, max(1, 8192 // gs))
        channels = gs * groups
        tokens = _log(rng, 1, min(32768, max(2, (1 << 26) // channels)))
        c = dict(op=op, tokens=tokens, channels=channels, dtype=dtype)
        if op != "save":
            c.update(groups=groups, gate=rng.choice(["first", "first", "last", "none"]),
                     center=rng.random() < 0.5, bias=rng.random() < 0.5,
                     pad=rng.choice([0, 0, 8, 8 * rng.randint(1, 700)]))
        if op == "norm_backward":
            c["ckpt"] = rng.random() < 0.5
        if op == "norm_save":
            c["pad"] = 0
        return c
    x_dim, bc_dim = 8 * _log(rng, 1, 640), 8 * _log(rng, 1, 128)
    ch = x_dim + 2 * bc_dim
    most = min(32768, (1 << 26) // ch)
    c = dict(op=op, batch=1, seqlen=0, num_seqs=0, max_len=0, len_seed=0, x_dim=x_dim,
             bc_dim=bc_dim, width=rng.choice([2, 3, 4, 4]), dtype=dtype,
             history=rng.random() < 0.5)
    if rng.random() < 0.5:
        c["batch"] = rng.randint(1, 8)
        c["seqlen"] = _log(rng, 1, max(2, most // c["batch"]))
    else:
        c["num_seqs"] = _log(rng, 1, 64)
        c["max_len"] = max(1, _log(rng, 2, max(2, most // c["num_seqs"])))
        c["len_seed"] = rng.randrange(1 << 20)
    if op == "conv_backward":
        c["ckpt"] = rng.random() < 0.5
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
    if op in ("norm", "norm_backward", "norm_save", "save"):
        n = case["tokens"] * case["channels"]
        q = n + case["tokens"] * -(-case["channels"] // BLOCK)     # one 8-bit copy
        gated = 0 if op == "save" or case["gate"] == "none" else 1
        wb = 0 if op == "save" else 4 * case["channels"] * (1 + case["bias"])
        if op == "save":
            return {"bytes": n * es * 2 + 2 * q, "flops": 6 * n}
        if op == "norm":
            return {"bytes": n * es * (2 + gated) + wb, "flops": 14 * n}
        if op == "norm_save":
            return {"bytes": n * es * (2 + gated) + wb + (1 + gated) * (2 * q + n * es),
                    "flops": 24 * n}
        src = (1 + gated) * (q if case["ckpt"] else n * es)
        return {"bytes": src + n * es * (2 + gated) + 2 * wb, "flops": 35 * n}
    lens = _lengths(case)
    ch, K = case["x_dim"] + 2 * case["bc_dim"], case["width"]
    n = sum(lens) * ch
    q = n + sum(lens) * -(-ch // BLOCK)
    hist = len(lens) * (K - 1) * ch * es
    taps = 4 * ch * (K + 1)
    given = hist if case["history"] else 0
    if op == "conv_save":
        return {"bytes": 2 * n * es + 2 * q + n * es + taps + hist + given, "flops": n * (2 * K + 10)}
    if op == "conv_load":
        return {"bytes": q + n * es + taps + given, "flops": n * (2 * K + 6)}
    return {"bytes": (q if case["ckpt"] else n * es) + 2 * n * es + 2 * taps + 2 * given,
            "flops": n * (6 * K + 12)}


# ---- inputs ------------------------------------------------------------------


def _uneven(g, rows, ch, dtype):
    """Activations as a layer makes them: channels of different sizes, a few rows far larger."""
    v = torch.randn(rows, ch, device="cuda", generator=g)
    v *= torch.exp(0.5 * torch.randn(1, ch, device="cuda", generator=g))
    v *= torch.exp(0.7 * torch.randn(rows, 1, device="cuda", generator=g))
    return v.to(dtype)


def _quantise(v):
    """(q int8, byte uint8) of rows of blocks: the step is the least power of two for which the
    block's largest value rounds to at most 127; the byte is its exponent + 127."""
    rows, ch = v.shape
    nb = -(-ch // BLOCK)
    f = v.float()
    if nb * BLOCK != ch:
        f = torch.cat([f, f.new_zeros(rows, nb * BLOCK - ch)], 1)
    f = f.view(rows, nb, BLOCK)
    m, e = torch.frexp(f.abs().amax(2))
    s = torch.where(torch.round(m * 128) <= 127, e - 7, e - 6)
    byte = (s + 127).clamp(min=2).to(torch.int32)
    q = torch.round(f / (byte << 23).view(torch.float32)[:, :, None])
    return q.to(torch.int8).view(rows, nb * BLOCK)[:, :ch].contiguous(), byte.to(torch.uint8)


def _values(q, byte):
    rows, ch = q.shape
    step = (byte.to(torch.int32) << 23).view(torch.float32)
    return q.float() * step.repeat_interleave(BLOCK, 1)[:, :ch]


def _inputs(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    if op == "save":
        return dict(case=case, x=_uneven(g, case["tokens"], case["channels"], dt))
    if op in ("norm", "norm_backward", "norm_save"):
        T, C = case["tokens"], case["channels"]
        s = dict(case=case, x=_uneven(g, T, C, dt), z=None, bias=None)
        s["weight"] = 1 + 0.1 * rand(C)
        if case["bias"]:
            s["bias"] = 0.1 * rand(C)
        if case["gate"] != "none":
            wide = rand(T, C + case["pad"]).to(dt)
            s["z"] = wide[:, :C]
        if op == "norm_backward":
            s["dout"] = (0.02 * rand(T, C)).to(dt)
            if case["ckpt"]:
                s["x"] = _quantise(s["x"])
                s["z"] = None if s["z"] is None else _quantise(s["z"])
        return s
    lens = _lengths(case)
    T, ch, K = sum(lens), case["x_dim"] + 2 * case["bc_dim"], case["width"]
    bound = 1 / math.sqrt(K)
    s = dict(case=case, xbc=_uneven(g, T, ch, dt), history=None, cu=None)
    s["weight"] = bound * (2 * torch.rand(ch, K, device="cuda", generator=g) - 1)
    s["bias"] = bound * (2 * torch.rand(ch, device="cuda", generator=g) - 1)
    if case["history"]:
        s["history"] = rand(len(lens), K - 1, ch).to(dt)
    ends = torch.tensor(lens, device="cuda").cumsum(0)
    cu = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    s["cu"] = cu if case["num_seqs"] else None
    if op == "conv_backward":
        s["dx"] = (0.02 * rand(T, case["x_dim"])).to(dt)
        s["dB"], s["dC"] = (0.1 * rand(2, T, case["bc_dim"])).to(dt)
    if op == "conv_load" or case.get("ckpt"):
        s["xbc"] = _quantise(s["xbc"])
    return s


def _dense(case, t):
    """A dense batch's view of token rows."""
    return t if case["num_seqs"] else t.view(case["batch"], case["seqlen"], t.shape[-1])


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import mamba_ssd_sequence_fwd_amd as ssd
        dt = DTYPES[case["dtype"]]
        s["ssd"] = ssd
        for k in ("x", "z", "xbc"):
            if isinstance(s.get(k), tuple):
                q, byte = s[k]
                if k == "xbc":
                    q, byte = _dense(case, q), _dense(case, byte)
                s[k] = ssd.Checkpoint(q, byte, dt)
            elif k == "xbc" and k in s:
                s[k] = _dense(case, s[k])
        for k in ("dx", "dB", "dC"):
            if k in s:
                s[k] = _dense(case, s[k])
    return s


# ---- the framework's operators -------------------------------------------------


def _run_own(s):
    c, ssd = s["case"], s["ssd"]
    op = c["op"]
    if op == "save":
        return ssd.checkpoint_save(s["x"]).load()
    if op in ("norm", "norm_backward", "norm_save"):
        kw = dict(groups=c["groups"], eps=EPS, center=c["center"],
                  norm_before_gate=c["gate"] == "last")
        if op == "norm":
            return ssd.group_norm_silu(s["x"], s["weight"], s["bias"], s["z"], **kw)
        if op == "norm_save":
            out, kx, kz = ssd.group_norm_silu(s["x"], s["weight"], s["bias"], s["z"],
                                              checkpoint=True, **kw)
            return [out, kx.load(), None if kz is None else kz.load()]
        g = ssd.group_norm_silu_backward(s["dout"], s["x"], s["weight"], s["bias"], s["z"], **kw)
        return [g["dx"], g["dz"], g["dweight"], g["dbias"] if c["bias"] else None]
    T = None if c["num_seqs"] else c["batch"] * c["seqlen"]

    def flat(t):
        return t if T is None else t.reshape(T, t.shape[-1])

    if op == "conv_backward":
        g = ssd.conv1d_silu_backward(s["xbc"], s["weight"], s["bias"], s["dx"], s["dB"], s["dC"],
                                     s["history"], s["cu"], check_cu_seqlens=False)
        return [flat(g["dxbc"]), g["dweight"], g["dbias"], g["dhistory"]]
    if op == "conv_save":
        x, B, C, hist, kept = ssd.conv1d_silu(s["xbc"], s["weight"], s["bias"], c["x_dim"],
                                              c["bc_dim"], s["history"], s["cu"],
                                              checkpoint=True, check_cu_seqlens=False)
        return [flat(x), flat(B), flat(C), hist, flat(kept.load())]
    x, B, C, _ = ssd.conv1d_silu(s["xbc"], s["weight"], s["bias"], c["x_dim"], c["bc_dim"],
                                 s["history"], s["cu"], check_cu_seqlens=False)
    return [flat(x), flat(B), flat(C)]


# ---- the plain forms ------------------------------------------------------------


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _plain_norm(s, backward):
    c = s["case"]
    dt, T, C, G = DTYPES[c["dtype"]], c["tokens"], c["channels"], c["groups"]
    wide = _values if c.get("ckpt") else (lambda t: t.float())
    x = wide(*s["x"]) if c.get("ckpt") else wide(s["x"])
    z = None if s["z"] is None else wide(*s["z"]) if c.get("ckpt") else wide(s["z"])
    w, b = s["weight"], s["bias"]
    sz = None if z is None else _sigmoid(z)
    u = x * (z * sz) if c["gate"] == "first" else x
    u = u.view(T, G, C // G)
    if c["center"]:
        u = u - u.mean(2, keepdim=True)
    r = 1 / torch.sqrt((u * u).mean(2, keepdim=True) + EPS)
    h = (u * r).view(T, C)
    v = h * w if b is None else h * w + b
    sv = _sigmoid(v) if c["gate"] == "none" else None
    if not backward:
        if c["gate"] == "last":
            v = v * (z * sz)
        elif c["gate"] == "none":
            v = v * sv
        return v.to(dt)
    d = s["dout"].float()
    if c["gate"] == "last":
        dv = d * (z * sz)
    elif c["gate"] == "none":
        dv = d * (sv * (1 + v * (1 - sv)))
    else:
        dv = d
    dw = (dv * h).sum(0, dtype=torch.float64).float()
    db = dv.sum(0, dtype=torch.float64).float() if b is not None else None
    g, hg = (dv * w).view(T, G, C // G), h.view(T, G, C // G)
    du = g - hg * (g * hg).mean(2, keepdim=True)
    if c["center"]:
        du = du - g.mean(2, keepdim=True)
    du = (du * r).view(T, C)
    if c["gate"] == "first":
        dx, dz = du * (z * sz), du * x * (sz * (1 + z * (1 - sz)))
    elif c["gate"] == "last":
        dx, dz = du, d * v * (sz * (1 + z * (1 - sz)))
    else:
        dx, dz = du, None
    return [dx.to(dt), None if dz is None else dz.to(dt), dw, db]


def _plain_conv(s, backward):
    c = s["case"]
    dt, K = DTYPES[c["dtype"]], c["width"]
    u = _values(*s["xbc"]) if isinstance(s["xbc"], tuple) else s["xbc"].float()
    T, ch = u.shape
    w, b = s["weight"], s["bias"]
    S = c["num_seqs"] or c["batch"]
    if s["cu"] is None:
        start = torch.arange(S + 1, device=u.device) * c["seqlen"]
    else:
        start = s["cu"].long()
    tok = torch.arange(T, device=u.device)
    seq = torch.searchsorted(start, tok, right=True) - 1
    pos, left = tok - start[seq], start[seq + 1] - tok - 1
    hist = s["history"].float() if s["history"] is not None else u.new_zeros(S, K - 1, ch)

    def before(k):
        """The input k tokens back: an earlier token of the sequence, or its history."""
        if k == 0:
            return u
        e = torch.empty_like(u)
        e[k:], e[:k] = u[:max(T - k, 0)], 0
        at = (pos < k).nonzero()[:, 0]
        e[at] = hist[seq[at], K - 1 - k + pos[at]]
        return e

    pre = b + w[:, K - 1] * u
    for k in range(1, K):
        pre = pre + w[:, K - 1 - k] * before(k)
    sp = _sigmoid(pre)
    if not backward:
        out = (pre * sp).to(dt)
        parts = list(out.split([c["x_dim"], c["bc_dim"], c["bc_dim"]], 1))
        if c["op"] == "conv_load":
            return parts
        last = torch.arange(K - 1, device=u.device)[None, :] + (start[1:] - start[:-1])[:, None]
        row = (start[:-1, None] + last - (K - 1)).clamp(0, T - 1)          # rows of [history; u]
        new = torch.where((last < K - 1)[:, :, None],
                          hist[torch.arange(S, device=u.device)[:, None], last.clamp(max=K - 2)],
                          u[row])
        return parts + [new.to(dt), _values(*_quantise(s["xbc"])).to(dt)]
    d = torch.cat([s["dx"], s["dB"], s["dC"]], 1).float()
    g = d * (sp * (1 + pre * (1 - sp)))
    du = w[:, K - 1] * g
    for k in range(1, K):
        later = torch.zeros_like(g)
        later[:max(T - k, 0)] = g[k:]
        later[left < k] = 0
        du = du + w[:, K - 1 - k] * later
    dw = torch.stack([(g * before(K - 1 - k)).sum(0, dtype=torch.float64) for k in range(K)], 1)
    db = g.sum(0, dtype=torch.float64)
    dh = None
    if s["history"] is not None:
        dh = u.new_zeros(S, K - 1, ch)
        length = start[1:] - start[:-1]
        for j in range(K - 1):
            for k in range(j + 1):
                at = (length > j - k).nonzero()[:, 0]
                dh[at, j] += w[:, k] * g[start[at] + (j - k)]
        dh = dh.to(dt)
    return [du.to(dt), dw.float(), db.float(), dh]


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    op = c["op"]
    if op == "save":
        return _values(*_quantise(state["x"])).to(DTYPES[c["dtype"]])
    if op == "norm":
        return _plain_norm(state, False)
    if op == "norm_save":
        out = _plain_norm(state, False)
        kept = [_values(*_quantise(t)).to(out.dtype) if t is not None else None
                for t in (state["x"], state["z"])]
        return [out] + kept
    if op == "norm_backward":
        return _plain_norm(state, True)
    return _plain_conv(state, op == "conv_backward")


# ---- from the definition, in 64 bits ----------------------------------------------


def _exact_values(v):
    """What 8 bits keep of v: multiples of a power of two of at most 127, the finest that hold
    each block of channels."""
    v = v.double()
    out = torch.empty_like(v)
    for c0 in range(0, v.shape[1], BLOCK):
        b = v[:, c0:c0 + BLOCK]
        top = b.abs().amax(1, keepdim=True)
        s = torch.full_like(top, -125.0)
        some = top > 0
        s[some] = torch.floor(torch.log2(top[some] / 127)) - 1
        for _ in range(3):
            s = torch.where(torch.round(top * torch.exp2(-s)) > 127, s + 1, s)
        s = s.clamp(min=-125)
        out[:, c0:c0 + BLOCK] = torch.round(b * torch.exp2(-s)) * torch.exp2(s)
    return out


def _kept(pair):
    q, byte = pair
    step = torch.exp2(byte.double() - 127)
    return q.double() * torch.repeat_interleave(step, BLOCK, 1)[:, :q.shape[1]]


def _exact_norm(s, r0, r1, grads):
    c = s["case"]

    def wide(t):
        return None if t is None else \
            _kept(tuple(p[r0:r1] for p in t)) if isinstance(t, tuple) else t[r0:r1].double()

    x, z = wide(s["x"]), wide(s["z"])
    w = s["weight"].double()
    b = torch.zeros_like(w) if s["bias"] is None else s["bias"].double()
    leaves = [t for t in (x, z, w, b) if t is not None]
    for t in leaves:
        t.requires_grad_(grads)
    u = x if c["gate"] != "first" else x * z * torch.sigmoid(z)
    rows = u.reshape((r1 - r0) * c["groups"], -1)
    if c["center"]:
        rows = rows - rows.sum(1, keepdim=True) / rows.shape[1]
    rows = rows * (rows.pow(2).sum(1, keepdim=True) / rows.shape[1] + EPS) ** -0.5
    v = rows.reshape(x.shape) * w + b
    if c["gate"] != "first":
        v = v * torch.sigmoid(v) if z is None else v * z * torch.sigmoid(z)
    if not grads:
        return v
    got = torch.autograd.grad(v, leaves, s["dout"][r0:r1].double())
    return list(got) if z is not None else [got[0], None, got[1], got[2]]


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "save":
        return _exact_values(s["x"])
    if op in ("norm", "norm_backward", "norm_save"):
        T, step = case["tokens"], max(1, (1 << 25) // case["channels"])
        parts = [_exact_norm(s, r, min(T, r + step), op == "norm_backward")
                 for r in range(0, T, step)]
        if op == "norm_backward":
            rows = [None if p[0] is None else torch.cat(p) for p in zip(*[q[:2] for q in parts])]
            return rows + [sum(q[2] for q in parts),
                           sum(q[3] for q in parts) if case["bias"] else None]
        out = torch.cat(parts)
        if op == "norm":
            return out
        return [out, _exact_values(s["x"]), None if s["z"] is None else _exact_values(s["z"])]
    K, ch = case["width"], case["x_dim"] + 2 * case["bc_dim"]
    split = [case["x_dim"], case["bc_dim"], case["bc_dim"]]
    w0, b0 = s["weight"].double(), s["bias"].double()
    outs, hists, at = [], [], 0
    dw, db = torch.zeros_like(w0), torch.zeros_like(b0)
    for k, n in enumerate(_lengths(case)):
        rows = slice(at, at + n)
        at += n
        u = _kept(tuple(p[rows] for p in s["xbc"])) if isinstance(s["xbc"], tuple) \
            else s["xbc"][rows].double()
        h = u.new_zeros(K - 1, ch) if s["history"] is None else s["history"][k].double()
        leaves = [t.clone().requires_grad_(op == "conv_backward") for t in (u, w0, b0, h)]
        u, w, b, h = leaves
        e = torch.cat([h, u])
        pre = b + sum(w[:, j] * e[j:j + n] for j in range(K))
        y = pre * torch.sigmoid(pre)
        if op == "conv_backward":
            d = torch.cat([s[p][rows] for p in ("dx", "dB", "dC")], 1).double()
            gu, gw, gb, gh = torch.autograd.grad(y, leaves, d)
            outs.append(gu)
            hists.append(gh)
            dw += gw
            db += gb
        else:
            outs.append(y)
            hists.append(e[n:])
    if op == "conv_backward":
        return [torch.cat(outs), dw, db, torch.stack(hists) if case["history"] else None]
    parts = list(torch.cat(outs).split(split, 1))
    if op == "conv_load":
        return parts
    return parts + [torch.stack(hists), _exact_values(s["xbc"])]
