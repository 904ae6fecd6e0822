"""The gated delta rule on the GPU (forward, backward, one-token step) against the
fp64 oracle; inputs and bounds in delta_helpers."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mamba_ssd_sequence_fwd_amd as ssd
from delta_helpers import BOUND, CASES, DT, STATE, backward, check, forward, inputs, on_gpu
from oracle.delta import delta_backward, delta_rule

pytestmark = pytest.mark.gpu
NAMES = list(CASES)
GRADS = ("dx", "dg", "dbeta", "dB", "dC")


def _wanted(d, case):
    return delta_rule(d["x"], d["g"], d["beta"], d["B"], d["C"], d["h0"], case[0])


def _wanted_grads(d, case):
    return delta_backward(d["x"], d["g"], d["beta"], d["B"], d["C"], d["h0"], case[0], d["dy"],
                          d["dhT"])


def _check_forward(d, t, cu, case):
    dtype = case[6]
    y, h = forward(t, cu)
    torch.cuda.synchronize()
    want, hw = _wanted(d, case)
    check("y", y, want, BOUND[dtype])
    check("final_state", h, hw, STATE[dtype])


def _check_backward(d, t, cu, case):
    dtype = case[6]
    g = backward(t, cu)
    torch.cuda.synchronize()
    want = _wanted_grads(d, case)
    for k in GRADS:
        check(k, g[k], want[k], BOUND[dtype])
    check("dinitial_state", g["dinitial_state"], want["dinitial_state"], STATE[dtype])


@pytest.mark.parametrize("name", NAMES)
def test_forward(name):
    case = CASES[name]
    d = inputs(case, 100 + NAMES.index(name))
    t, cu = on_gpu(d, case)
    print("[gpu] delta forward %s" % name, flush=True)
    _check_forward(d, t, cu, case)


@pytest.mark.parametrize("name", NAMES)
def test_backward(name):
    case = CASES[name]
    d = inputs(case, 200 + NAMES.index(name))
    t, cu = on_gpu(d, case)
    print("[gpu] delta backward %s" % name, flush=True)
    _check_backward(d, t, cu, case)


@pytest.mark.parametrize("name", ["packed", "segments", "packed-fp32", "one-chunk-and-one"])
@pytest.mark.parametrize("what", ["reflections", "strong-decay", "no-decay", "resets"])
def test_gates(name, what):
    """beta near 2 (each write reflects), g far below and at zero, and g = -inf, which
    forgets all before it."""
    case = CASES[name]
    d = inputs(case, 300 + NAMES.index(name), rate=40.0 if what == "strong-decay" else
               0.0 if what == "no-decay" else 0.2, top=2.0 if what == "reflections" else 1.0)
    if what == "resets":
        d["g"][::37, 0] = -float("inf")
        d["g"][5, 1] = -1000.0
    t, cu = on_gpu(d, case)
    print("[gpu] delta gates %s %s" % (name, what), flush=True)
    _check_forward(d, t, cu, case)
    if what == "resets":
        # exp(-inf) has no derivative that differences could show: the formula's is zero
        d["g"] = d["g"].clamp_min(-1e5)
    _check_backward(d, t, cu, case)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_equal_keys(dtype):
    """One key for all tokens of a chunk (the triangular system at its worst), and
    keys of length zero."""
    case = ([130, 130], False, 4, 64, 64, 1, dtype, True)
    d = inputs(case, 400, top=1.0)
    d["B"][:] = d["B"][:1]
    d["B"][140:200] = 0
    t, cu = on_gpu(d, case)
    print("[gpu] delta equal keys %s" % dtype, flush=True)
    _check_forward(d, t, cu, case)
    _check_backward(d, t, cu, case)


@pytest.mark.parametrize("name", ["packed", "segments", "packed-fp32", "P128-N256"])
def test_gradients_without_states(name):
    """No initial state and no gradient of the final one; what is not asked for is
    not needed."""
    case = CASES[name][:7] + (False,)
    d = inputs(case, 500)
    t, cu = on_gpu(d, case)
    print("[gpu] delta without states %s" % name, flush=True)
    _check_backward(d, t, cu, case)
    y, h = forward(t, cu, want_final_state=False)
    assert h is None and torch.equal(y, forward(t, cu)[0])


def test_gradients_are_differences():
    """The fp32 gradients against central differences of the fp32 forward call along
    random directions: step 2^-6, so the truncation is 2^-12 / 6 of a third derivative
    of the loss' size and the rounding 2^-24 * 2^6 of the loss' terms' norm: 1e-3 of
    the largest directional derivative holds both."""
    case = ([70, 70], False, 2, 16, 16, 1, "fp32", True)
    d = inputs(case, 600)
    t, cu = on_gpu(d, case)
    print("[gpu] delta differences", flush=True)
    g = backward(t, cu)

    def loss(**kw):
        y, h = forward(dict(t, **kw), cu)
        return float((y.double() * t["dy"].double()).sum() + (h.double() * t["dhT"].double()).sum())

    rng = torch.Generator().manual_seed(1)
    step = 2.0 ** -6
    for k, grad in (("x", "dx"), ("g", "dg"), ("beta", "dbeta"), ("B", "dB"), ("C", "dC"),
                    ("h0", "dinitial_state")):
        v = torch.randn(t[k].shape, generator=rng).cuda()
        v /= v.norm()
        got = float((g[grad].double() * v.double()).sum())
        want = (loss(**{k: t[k] + step * v}) - loss(**{k: t[k] - step * v})) / (2 * step)
        assert abs(got - want) <= 1e-3 * float(g[grad].double().norm()), (k, got, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes", [(1, 24, 64, 128, 1), (5, 6, 16, 48, 3), (3, 4, 128, 256, 2),
                                   (7, 5, 32, 16, 5), (2, 3, 128, 80, 1)])
def test_steps(dtype, sizes):
    """Tokens one at a time, the state in place: the oracle's, and the forward call's
    final state. y: two products of fp32 values, rounded once."""
    S, H, P, N, G = sizes
    T = 9
    case = ([T] * S, False, H, P, N, G, dtype, True)
    d = inputs(case, 700 + H)
    t, cu = on_gpu(d, case)
    print("[gpu] delta steps %s %s" % (sizes, dtype), flush=True)
    state = t["h0"].clone()
    ys = [ssd.delta_step(t["x"][:, k], t["g"][:, k], t["beta"][:, k], t["B"][:, k], t["C"][:, k],
                         state) for k in range(T)]
    torch.cuda.synchronize()
    want, hw = _wanted(d, case)
    check("y", torch.stack(ys, 1), want, 2.0 ** -8 if dtype == "bf16" else BOUND["fp32"])
    check("state", state, hw, STATE["fp32"])
    check("final_state", forward(t, cu)[1], hw, STATE[dtype])


def test_step_takes_slices_and_outputs():
    case = ([1] * 6, False, 4, 64, 64, 2, "bf16", True)
    d = inputs(case, 800)
    t, _ = on_gpu(d, case)
    one = {k: t[k][:, 0] for k in ("x", "g", "beta", "B", "C")}
    s0, s1 = t["h0"].clone(), t["h0"].clone()
    want = ssd.delta_step(one["x"], one["g"], one["beta"], one["B"], one["C"], s0)
    wide = {k: torch.randn((6, v.shape[1] + 3) + v.shape[2:], device="cuda").to(v.dtype)
            for k, v in one.items()}
    for k, v in one.items():
        wide[k][:, 1:-2] = v
        one[k] = wide[k][:, 1:-2]
    out = torch.empty_like(want)
    print("[gpu] delta step slices", flush=True)
    assert ssd.delta_step(one["x"], one["g"], one["beta"], one["B"], one["C"], s1, y=out) is out
    assert torch.equal(out, want) and torch.equal(s0, s1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_slices_and_outputs(dtype):
    """Inputs that are slices of wider rows (as the convolution front gives them) or
    start off 16 bytes, and the caller's outputs: the same bits."""
    case = ([90, 90], False, 4, 32, 48, 2, dtype, True)
    d = inputs(case, 900)
    t, cu = on_gpu(d, case)
    want, hw = forward(t, cu)
    gw = backward(t, cu)
    s = dict(t)
    for k in ("x", "B", "C", "g", "beta", "dy"):
        v = t[k]
        wide = torch.full((2, 90, v[0, 0].numel() + 9), float("nan"), device="cuda", dtype=v.dtype)
        wide[..., 1:-8] = v.flatten(2)
        s[k] = wide[..., 1:-8].unflatten(2, v.shape[2:])
    for k in ("h0", "dhT"):
        flat = torch.empty(t[k].numel() + 1, device="cuda")
        flat[1:] = t[k].flatten()
        s[k] = flat[1:].view(t[k].shape)
    y, h = torch.empty_like(want), torch.empty_like(hw)
    print("[gpu] delta slices %s" % dtype, flush=True)
    assert forward(s, cu, y=y, final_state=h)[0] is y
    assert torch.equal(y, want) and torch.equal(h, hw)
    g = backward(s, cu)
    assert all(torch.equal(g[k], gw[k]) for k in gw)


def test_without_tokens():
    """Sequences of no tokens hand their states through."""
    z = lambda *s: torch.zeros(s, device="cuda", dtype=torch.bfloat16)
    h0 = torch.randn(2, 4, 64, 32, device="cuda")
    print("[gpu] delta without tokens", flush=True)
    args = (z(2, 0, 4, 64), z(2, 0, 4), z(2, 0, 4), z(2, 0, 1, 32), z(2, 0, 1, 32))
    y, h = ssd.delta_forward(*args, h0)
    assert y.shape == (2, 0, 4, 64) and torch.equal(h, h0)
    g = ssd.delta_backward(*args, h0, z(2, 0, 4, 64), 2 * h0)
    assert torch.equal(g["dinitial_state"], 2 * h0) and g["dx"].numel() == 0
    y, h = ssd.delta_forward(*args)
    assert torch.equal(h, torch.zeros_like(h0))
    none = (z(0, 5, 4, 64), z(0, 5, 4), z(0, 5, 4), z(0, 5, 1, 32), z(0, 5, 1, 32))
    assert ssd.delta_forward(*none)[1].shape == (0, 4, 64, 32)
    assert ssd.delta_backward(*none, None, none[0])["dB"].numel() == 0
    assert ssd.delta_step(*(v[:, 0] for v in none), h0[:0]).numel() == 0


def test_sequences_do_not_see_each_other():
    """NaN in one sequence of a packed batch stays in it, whatever chunk or segment
    its neighbours end in."""
    for name in ("packed", "segments-packed", "packed-fp32"):
        case = CASES[name]
        d = inputs(case, 1000)
        t, cu = on_gpu(d, case)
        want, hw = forward(t, cu)
        gw = backward(t, cu)
        bad = int(np.argmax(case[0]))
        a, b = int(cu[bad]), int(cu[bad + 1])
        s = {k: v.clone() for k, v in t.items()}
        for k in ("x", "g", "beta", "B", "C", "dy"):
            s[k][0, a:b] = float("nan")
        print("[gpu] delta NaN in a neighbour, %s" % name, flush=True)
        y, h = forward(s, cu)
        g = backward(s, cu)
        keep = torch.ones(y.shape[1], dtype=torch.bool)
        keep[a:b] = False
        keep = keep.cuda()
        assert y[0, a:b].isnan().all()
        assert torch.equal(y[0, keep], want[0, keep])
        assert all(torch.equal(g[k][0, keep], gw[k][0, keep]) for k in GRADS)
        others = [i for i in range(len(case[0])) if i != bad]
        assert torch.equal(h[others], hw[others])
        assert torch.equal(g["dinitial_state"][others], gw["dinitial_state"][others])


def test_what_fits_no_32_bits():
    """x and y of 2^31 elements and more: the last sequences are those of a call of
    their own."""
    H, P, N, L, S = 64, 128, 16, 1088, 242
    case = ([L] * 2, False, H, P, N, 1, "bf16", False)
    d = inputs(case, 1100)
    t, _ = on_gpu(d, case)
    assert S * L * H * P > 1 << 31
    big = {k: v[:1].expand((S,) + v.shape[1:]).contiguous() for k, v in t.items()}
    for k, v in t.items():
        big[k][-2:] = v
    print("[gpu] delta with %d values" % big["x"].numel(), flush=True)
    y, h = forward(big, None)
    want, hw = _wanted(d, case)
    check("y", y[-2:], want, BOUND["bf16"])
    check("final_state", h[-2:], hw, STATE["bf16"])
    assert torch.equal(y[:-2], y[:1].expand_as(y[:-2]))


@pytest.mark.parametrize("name", ["packed", "segments", "packed-fp32"])
def test_equal_calls_give_equal_bits(name):
    case = CASES[name]
    t, cu = on_gpu(inputs(case, 1200), case)
    print("[gpu] delta twice %s" % name, flush=True)
    a, b = forward(t, cu), forward(t, cu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = backward(t, cu), backward(t, cu)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_two_streams():
    """Calls on two streams at once, with workspaces of their own: the bits of calls
    one after the other."""
    case = CASES["segments-N128"]
    ts = [on_gpu(inputs(case, 1300 + i), case)[0] for i in range(2)]
    want = [(forward(t, None), backward(t, None)) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    print("[gpu] delta on two streams", flush=True)
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            got[i].append((forward(ts[i], None, stream=s), backward(ts[i], None, stream=s)))
    torch.cuda.synchronize()
    for i in range(2):
        for f, b in got[i]:
            assert torch.equal(f[0], want[i][0][0]) and torch.equal(f[1], want[i][0][1])
            assert all(torch.equal(b[k], want[i][1][k]) for k in b)


@pytest.mark.parametrize("name", ["packed", "segments", "packed-fp32"])
def test_captured(name):
    """Forward, backward and a step in one graph, replayed on new inputs with eager
    work between; and a second graph of the same sizes, replayed in turn."""
    case = CASES[name]
    d = [inputs(case, 1400 + i) for i in range(3)]
    t, cu = on_gpu(d[0], case)
    cu = cu.cuda() if cu is not None else None
    new = [on_gpu(v, case)[0] for v in d]
    kw = dict(check_cu_seqlens=False)

    def work(v):
        f, b = forward(v, cu, **kw), backward(v, cu, **kw)
        state = v["h0"].clone()
        tok = lambda k: v[k][0, :state.shape[0]]
        y = ssd.delta_step(tok("x"), tok("g"), tok("beta"), tok("B"), tok("C"), state)
        return [f[0], f[1], state, y] + [b[k] for k in b]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(t)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    print("[gpu] delta captured %s" % name, flush=True)
    graphs = []
    for _ in range(2):
        v = {k: w.clone() for k, w in t.items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = work(v)
        graphs.append((graph, v, out))
    for r in range(6):
        graph, v, out = graphs[r % 2]
        for k in v:
            v[k].copy_(new[r % 3][k])
        graph.replay()
        want = work(new[r % 3])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), r


def test_device_offsets_need_no_check():
    case = CASES["packed"]
    t, cu = on_gpu(inputs(case, 1500), case)
    want = forward(t, cu)
    print("[gpu] delta device offsets", flush=True)
    for c in (cu.cuda(), cu.long().cuda()):
        got = forward(t, c, check_cu_seqlens=False)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_values_that_are_not_finite(dtype):
    """An infinite value stays in its channel and sequence and does not reach an
    earlier chunk; a NaN gate or key makes all that follows NaN."""
    case = ([200, 90, 90], True, 2, 32, 48, 1, dtype, False)
    d = inputs(case, 1600)
    t, cu = on_gpu(d, case)
    want, hw = forward(t, cu)
    s = dict(t, x=t["x"].clone())
    s["x"][0, 150, 1, 5] = float("inf")
    print("[gpu] delta not finite %s" % dtype, flush=True)
    y, h = forward(s, cu)
    assert not y[0, 150:200, 1, 5].isfinite().any()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[0, 128:200, 1, 5] = False
    assert torch.equal(y[keep], want[keep])
    hk = torch.ones_like(h, dtype=torch.bool)
    hk[0, 1, 5] = False
    assert torch.equal(h[hk], hw[hk])
    for k in ("g", "B"):
        s = dict(t)
        s[k] = t[k].clone()
        s[k][0, 70] = float("nan")
        y, h = forward(s, cu)
        assert y[0, 70:200].isnan().all() and h[0].isnan().all()
        assert torch.equal(y[0, :64], want[0, :64]) and torch.equal(y[0, 200:], want[0, 200:])
        assert torch.equal(h[1:], hw[1:])
