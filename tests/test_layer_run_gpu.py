"""The operators around the SSD layer run together, as a training step and a
decoding loop use them, on the GPU against the fp64 oracle chain: the
convolution front, the layer, the norm and gate, and their backward passes
from 8-bit checkpoints. Normwise bounds of the SSD parity tests (the chain
rounds every tensor between two operators to bf16)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mamba_ssd_sequence_fwd_amd as ssd
import oracle
import ssd_inputs as si
from gpu_helpers import TOL, rel_err
from oracle.backward import ssd_backward
from oracle.checkpoint import kept
from oracle.conv import conv_front, dense_bounds, varlen_bounds
from oracle.conv_backward import conv_backward
from oracle.norm import norm, norm_backward

pytestmark = pytest.mark.gpu

H, P, G, N, K = 4, 64, 1, 64, 4
X, BC = H * P, G * N
CH = X + 2 * BC


def _inputs(lens, seed, packed):
    """Rows of one projection output [z | xBC | dt], weights and a gradient."""
    rng = np.random.default_rng(seed)
    T = sum(lens)
    proj = torch.from_numpy(rng.standard_normal((T, X + CH + 8)).astype(np.float32)).to(torch.bfloat16)
    w = si.make_conv_inputs(1, 1, X, BC, K, "bf16", seed=seed + 1)
    p = dict(proj=proj, cw=w["weight"], cb=w["bias"],
             A=torch.from_numpy(-np.exp(rng.uniform(0, 2, H)).astype(np.float32)),
             D=torch.from_numpy(rng.standard_normal(H).astype(np.float32)),
             nw=torch.from_numpy((1 + 0.1 * rng.standard_normal(X)).astype(np.float32)),
             dt=torch.nn.functional.softplus(proj[:, X + CH:X + CH + H].float() - 2).to(torch.bfloat16),
             dout=torch.from_numpy(rng.standard_normal((T, X)).astype(np.float32)).to(torch.bfloat16))
    p["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32) if packed else None
    p["lens"] = lens
    return p


class Step:
    """One training step's forward and backward on device copies of the inputs."""

    def __init__(self, p):
        self.p = {k: v.cuda() if isinstance(v, torch.Tensor) and k != "cu" else v for k, v in p.items()}
        self.cu = p["cu"]
        if self.cu is not None:
            self.cu = self.cu.cuda()
        self.lead = (1, p["proj"].shape[0]) if self.cu is not None else (len(p["lens"]), p["lens"][0])

    def run(self):
        p, lead = self.p, self.lead
        T = p["proj"].shape[0]
        rows = (T,) if self.cu is not None else lead
        z = p["proj"][:, :X]
        xbc = p["proj"][:, X:X + CH].view(*rows, CH)
        kw = dict(check_cu_seqlens=False) if self.cu is not None else {}
        x, B, C, _, k_xbc = ssd.conv1d_silu(xbc, p["cw"], p["cb"], X, BC, None, self.cu,
                                            checkpoint=True, **kw)
        v = lambda x, B, C: (x.view(*lead, H, P), p["dt"].view(*lead, H), p["A"],
                             B.view(*lead, G, N), C.view(*lead, G, N), p["D"])
        y, _ = ssd.Plan(*v(x, B, C), chunk_size=128, cu_seqlens=self.cu, check_cu_seqlens=False).run()
        out, k_y, k_z = ssd.group_norm_silu(y.view(T, X), p["nw"], None, z, groups=2,
                                            checkpoint=True)
        del x, B, C, y                       # what a training step lets go of
        # backward, from the three checkpoints; the projection's gradient in place
        dproj = torch.zeros_like(p["proj"])
        gn = ssd.group_norm_silu_backward(p["dout"], k_y, p["nw"], None, k_z, groups=2,
                                          dz=dproj[:, :X])
        x, B, C, _ = ssd.conv1d_silu(k_xbc, p["cw"], p["cb"], X, BC, None, self.cu, **kw)
        gs = ssd.BackwardPlan(*v(x, B, C), None, gn["dx"].view(*lead, H, P), chunk_size=128,
                              cu_seqlens=self.cu, check_cu_seqlens=False).run()
        f = lambda t: t.reshape(*rows, *t.shape[2:])
        gc = ssd.conv1d_silu_backward(k_xbc, p["cw"], p["cb"], f(gs["dx"]), f(gs["dB"]),
                                      f(gs["dC"]), None, self.cu,
                                      dxbc=dproj[:, X:X + CH].view(*rows, CH), **kw)
        return dict(out=out, dproj=dproj, ddt=gs["ddt"].reshape(T, H), dA=gs["dA"], dD=gs["dD"],
                    dnw=gn["dweight"], dcw=gc["dweight"], dcb=gc["dbias"])


def _reference(p):
    """The same in fp64, with the checkpoints' values where they are read."""
    f = oracle._np
    lens, T = p["lens"], p["proj"].shape[0]
    bounds = varlen_bounds(p["cu"].tolist()) if p["cu"] is not None else dense_bounds(len(lens), lens[0])
    z, xbc = f(p["proj"][:, :X]), f(p["proj"][:, X:X + CH])

    def layer(x, B, C):
        return (x.reshape(T, H, P), f(p["dt"]), f(p["A"]), B.reshape(T, G, N), C.reshape(T, G, N),
                f(p["D"]))

    x, B, C, _ = conv_front(xbc, p["cw"], p["cb"], bounds, X, BC)
    y, _ = oracle.ssd_recurrence(*layer(x, B, C), None, lens)
    y = y.reshape(T, X)
    args = (2, 1e-5, False, "first")
    out, _ = norm(y, z, p["nw"], None, *args)
    gn, _ = norm_backward(p["dout"], kept(torch.from_numpy(y).to(torch.bfloat16)), kept(z), p["nw"],
                          None, *args)
    xk = kept(xbc)
    x, B, C, _ = conv_front(xk, p["cw"], p["cb"], bounds, X, BC)
    gs = ssd_backward(*layer(x, B, C), None, lens, gn["dx"].reshape(T, H, P), None)
    d = np.concatenate([gs["dx"].reshape(T, X), gs["dB"].reshape(T, BC), gs["dC"].reshape(T, BC)], 1)
    gc, _ = conv_backward(xk, p["cw"], p["cb"], bounds, d)
    return dict(out=out, dproj=np.concatenate([gn["dz"], gc["dxbc"], np.zeros((T, 8))], 1),
                ddt=gs["ddt"], dA=gs["dA"], dD=gs["dD"], dnw=gn["dweight"], dcw=gc["dweight"],
                dcb=gc["dbias"])


@pytest.mark.parametrize("lens,packed", [([150, 150], False), ([5, 0, 200, 1, 130], True)])
def test_training_step(lens, packed):
    p = _inputs(lens, 61, packed)
    print("[gpu] training step %s" % lens, flush=True)
    got = Step(p).run()
    torch.cuda.synchronize()
    want = _reference(p)
    for k, v in want.items():
        e = rel_err(got[k].double().cpu().numpy().reshape(v.shape), v)
        print("  %-6s err %.2e" % (k, e), flush=True)
        assert e <= TOL["bf16"], (k, e)


def test_training_step_captured():
    """The step captured into a graph and replayed, with eager work and new
    inputs in between: every replay equals the eager step."""
    p = _inputs([150, 150], 62, False)
    step = Step(p)
    print("[gpu] training step captured", flush=True)
    step.run()                                # warm up outside the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step.run()
    for seed in (62, 63, 64):
        q = _inputs([150, 150], seed, False)
        for k in ("proj", "dout", "dt"):
            step.p[k].copy_(q[k])
        eager = step.run()
        graph.replay()
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(held[k], eager[k]), (seed, k)


def test_decoding_follows_the_sequence():
    """A prompt and then token by token (front with its history, decode step,
    norm and gate), against the whole sequence at once in fp64."""
    L, first, S = 40, 33, 3
    p = _inputs([L] * S, 65, False)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    proj, dt = d["proj"].view(S, L, -1), d["dt"].view(S, L, H)
    print("[gpu] decoding loop", flush=True)

    def front(a, e, hist):
        return ssd.conv1d_silu(proj[:, a:e, X:X + CH].contiguous(), d["cw"], d["cb"], X, BC, hist)

    x, B, C, hist = front(0, first, None)
    y, state = ssd.forward(x.view(S, first, H, P), dt[:, :first], d["A"], B.view(S, first, G, N),
                           C.view(S, first, G, N), d["D"], chunk_size=128)
    outs = [ssd.group_norm_silu(y.view(S, first, X), d["nw"], None, proj[:, :first, :X], groups=2)]
    for t in range(first, L):
        x, B, C, hist = front(t, t + 1, hist)
        y = ssd.step(x.view(S, H, P), dt[:, t].contiguous(), d["A"], B.view(S, G, N),
                     C.view(S, G, N), d["D"], state)
        outs.append(ssd.group_norm_silu(y.view(S, X), d["nw"], None, proj[:, t, :X],
                                        groups=2).view(S, 1, X))
    torch.cuda.synchronize()
    want = _reference(p)["out"].reshape(S, L, X)
    got = torch.cat(outs, 1).double().cpu().numpy()
    for name, a, e in (("prompt", 0, first), ("tokens", first, L)):
        err = rel_err(got[:, a:e], want[:, a:e])
        print("  %s err %.2e" % (name, err), flush=True)
        assert err <= TOL["bf16"], (name, err)


def test_two_graphs_and_two_streams():
    """Two captured norm backward passes, and two streams at once: each call
    has outputs and a workspace of its own."""
    rng = np.random.default_rng(66)
    t = lambda: torch.from_numpy(rng.standard_normal((300, 640)).astype(np.float32)).to(torch.bfloat16).cuda()
    sets = [(t(), t(), t()) for _ in range(2)]
    w = torch.ones(640, device="cuda")
    call = lambda s, **kw: ssd.group_norm_silu_backward(s[0], s[1], w, None, s[2], **kw)
    print("[gpu] two graphs, two streams", flush=True)
    want = [call(s) for s in sets]
    torch.cuda.synchronize()
    graphs, held = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(call(s))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        again = [call(s) for s in sets]
        torch.cuda.synchronize()
        for a, b, c in zip(held, again, want):
            for k in ("dx", "dz", "dweight"):
                assert torch.equal(a[k], c[k]) and torch.equal(b[k], c[k]), k
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[call(s, stream=st) for _ in range(5)] for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for many, c in zip(got, want):
        for a in many:
            for k in ("dx", "dz", "dweight"):
                assert torch.equal(a[k], c[k]), k
