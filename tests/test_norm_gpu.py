"""Group norm with SiLU (ssd_group_norm_silu and its backward pass) on the GPU
against the fp64 oracle; bounds in layer_helpers."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import mamba_ssd_sequence_fwd_amd as ssd
from layer_helpers import DT, check, rows
from oracle.checkpoint import kept, quantise
from oracle.norm import norm, norm_backward

pytestmark = pytest.mark.gpu

CASES = {
    # name: (tokens, channels, groups, dtype, gate, center, affine, z pad)
    "one-token-2.7b": (1, 5120, 1, "bf16", "first", False, "w", 5456),
    "rows-2.7b": (37, 5120, 1, "bf16", "first", False, "w", 5456),
    "groups-of-512": (65, 4096, 8, "bf16", "first", False, "w", 0),
    "groups-of-8-fp32": (7, 64, 8, "fp32", "last", True, "wb", 8),
    "groups-of-24": (33, 120, 5, "bf16", "last", False, "", 16),
    "groups-of-40-center": (130, 200, 5, "bf16", "first", True, "wb", 0),
    "per-head-fp32": (99, 1536, 24, "fp32", "last", True, "wb", 0),
    "one-group-of-8": (3, 8, 1, "fp32", "none", True, "wb", 0),
    "no-gate-fp32": (41, 1280, 4, "fp32", "none", True, "wb", 0),
    "no-gate-bf16": (17, 520, 1, "bf16", "none", False, "b", 0),
    "wide-two-groups": (5, 2080, 2, "bf16", "last", True, "w", 24),
    "last-in-1024-lanes": (9, 8192, 1, "fp32", "first", True, "wb", 0),
    "two-parts-a-lane": (6, 8200, 1, "bf16", "first", False, "wb", 0),
    "widest-fp32": (3, 16384, 1, "fp32", "last", True, "wb", 0),
    "widest-no-gate": (4, 16384, 1, "bf16", "none", True, "", 0),
    "more-rows-than-blocks": (5000, 128, 2, "bf16", "first", False, "w", 0),
}


def _inputs(name):
    T, C, G, dtype, gate, center, affine, pad = CASES[name]
    rng = np.random.default_rng(100 + sorted(CASES).index(name))
    x, xn = rows(rng, T, C, dtype, pad=8 if pad else 0)
    z = zn = None
    if gate != "none":
        z, zn = rows(rng, T, C, dtype, pad=pad, spread=0.0)
    d, dn = rows(rng, T, C, dtype)
    w = (1 + 0.2 * rng.standard_normal(C)).astype(np.float32) if "w" in affine else None
    b = (0.2 * rng.standard_normal(C)).astype(np.float32) if "b" in affine else None
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()
    kw = dict(groups=G, eps=1e-5, center=center, norm_before_gate=gate == "last")
    return dict(x=x, z=z, d=d, w=dev(w), b=dev(b), kw=kw, dtype=dtype), \
        dict(x=xn, z=zn, d=dn, w=w, b=b, args=(G, 1e-5, center, gate))


@pytest.mark.parametrize("name", sorted(CASES))
def test_norm_forward(name):
    t, n = _inputs(name)
    print("[gpu] group norm %s" % name, flush=True)
    out = ssd.group_norm_silu(t["x"], t["w"], t["b"], t["z"], **t["kw"])
    torch.cuda.synchronize()
    want, size = norm(n["x"], n["z"], n["w"], n["b"], *n["args"])
    check("out", out, want, size, t["dtype"], 160)


@pytest.mark.parametrize("name", sorted(CASES))
def test_norm_backward(name):
    t, n = _inputs(name)
    print("[gpu] group norm backward %s" % name, flush=True)
    g = ssd.group_norm_silu_backward(t["d"], t["x"], t["w"], t["b"], t["z"], **t["kw"])
    torch.cuda.synchronize()
    want, size = norm_backward(n["d"], n["x"], n["z"], n["w"], n["b"], *n["args"])
    assert (g["dz"] is None) == (t["z"] is None)
    for k in ("dx", "dz", "dweight", "dbias"):
        if g[k] is not None:
            check(k, g[k], want[k], size[k], "fp32" if k in ("dweight", "dbias") else t["dtype"],
                  512)
    assert (g["dweight"] is None) == (t["w"] is None)
    assert (g["dbias"] is None) == (t["b"] is None)


@pytest.mark.parametrize("name", sorted(CASES))
def test_norm_checkpoints(name):
    """Saved on the way: bit for bit the oracle's 8 bits, the output unchanged;
    and the backward pass from them is that at their values."""
    t, n = _inputs(name)
    print("[gpu] group norm checkpoints %s" % name, flush=True)
    plain = ssd.group_norm_silu(t["x"], t["w"], t["b"], t["z"], **t["kw"])
    out, kx, kz = ssd.group_norm_silu(t["x"], t["w"], t["b"], t["z"], checkpoint=True, **t["kw"])
    g = ssd.group_norm_silu_backward(t["d"], kx, t["w"], t["b"], kz, **t["kw"])
    torch.cuda.synchronize()
    assert torch.equal(out, plain)
    for k, v in ((kx, n["x"]), (kz, n["z"])):
        assert (k is None) == (v is None)
        if k is not None:
            q, byte = quantise(v)
            assert np.array_equal(k.q.cpu().numpy(), q)
            assert np.array_equal(k.exponents.cpu().numpy(), byte)
    xk, zk = kept(n["x"]), None if n["z"] is None else kept(n["z"])
    want, size = norm_backward(n["d"], xk, zk, n["w"], n["b"], *n["args"])
    for k in ("dx", "dz", "dweight", "dbias"):
        if g[k] is not None:
            check(k, g[k], want[k], size[k], "fp32" if k in ("dweight", "dbias") else t["dtype"],
                  512)


def test_norm_gradients_are_differences():
    """dx and dz of the fp32 kernels against central differences of the fp32
    forward kernel: h = 2^-7, so the truncation h^2/6 |f'''| and the rounding
    (2^-24 of out, times the 8-channel group, over h) both stay under 2e-3."""
    rng = np.random.default_rng(3)
    T, C = 2, 8
    x, z, d = (torch.from_numpy(rng.standard_normal((T, C)).astype(np.float32)).cuda()
               for _ in range(3))
    w = torch.ones(C, device="cuda")
    print("[gpu] group norm differences", flush=True)
    for kw in (dict(), dict(center=True), dict(norm_before_gate=True)):
        kw = dict(eps=0.5, **kw)
        g = ssd.group_norm_silu_backward(d, x, w, None, z, **kw)
        for name, v in (("dx", x), ("dz", z)):
            for i in range(T):
                for j in range(C):
                    keep = float(v[i, j])
                    f = []
                    for h in (2.0 ** -7, -2.0 ** -7):
                        v[i, j] = keep + h
                        f.append(float((ssd.group_norm_silu(x, w, None, z, **kw).double()
                                        * d.double()).sum()))
                    v[i, j] = keep
                    diff = (f[0] - f[1]) * 2.0 ** 6
                    assert abs(diff - float(g[name][i, j])) < 2e-3, (kw, name, i, j)


def test_norm_special_values():
    """A zero row gives the bias (and zero gradients of the gate); infinities
    and NaN stay in their token's group; the checkpoint marks their blocks."""
    C = 128
    rng = np.random.default_rng(4)
    x, _ = rows(rng, 4, C, "bf16")
    z, _ = rows(rng, 4, C, "bf16")
    x, z = x.contiguous(), z.contiguous()
    clean = ssd.group_norm_silu(x, None, None, z, groups=2)
    x[0] = 0
    x[1, 3], x[2, 70] = float("nan"), float("inf")
    b = torch.randn(C, device="cuda")
    print("[gpu] group norm special values", flush=True)
    out, kx, kz = ssd.group_norm_silu(x, None, None, z, groups=2, checkpoint=True)
    outb = ssd.group_norm_silu(x, None, b, z, groups=2)
    g = ssd.group_norm_silu_backward(torch.ones_like(x), kx, None, b, kz, groups=2)
    torch.cuda.synchronize()
    assert torch.count_nonzero(out[0]) == 0 and torch.equal(outb[0], b.to(torch.bfloat16))
    assert torch.isnan(out[1, :64]).all() and torch.equal(out[1, 64:], clean[1, 64:])
    assert torch.equal(out[2, :64], clean[2, :64]) and not torch.isfinite(out[2, 64:]).all()
    assert torch.equal(out[3], clean[3])
    assert kx.exponents[1].tolist()[0] == 255 and kx.exponents[2].tolist()[2] == 255
    assert torch.isnan(g["dx"][1, :64]).all() and torch.isfinite(g["dx"][1, 64:]).all()
    assert torch.isfinite(g["dx"][3]).all() and torch.count_nonzero(g["dz"][0]) == 0


@pytest.mark.parametrize("C,G,ckpt", [
    (120, 5, False), (24, 3, False), (1040, 2, False), (1040, 2, True), (280, 7, True),
    (8704, 2, False), (8704, 2, True),
])
def test_norm_groups_do_not_see_each_other(C, G, ckpt):
    """Groups that leave lanes over: NaN and infinities in the first group (and
    in its weights) change no bit of the others, forward and backward."""
    rng = np.random.default_rng(9)
    T, gs = 5, C // G
    x, z, d = (rows(rng, T, C, "bf16")[0] for _ in range(3))
    w, b = torch.randn(C, device="cuda"), torch.randn(C, device="cuda")
    print("[gpu] group norm between groups %d/%d" % (C, G), flush=True)

    def both(**kw):
        zz = None if kw.pop("none", False) else z
        out, kx, kz = ssd.group_norm_silu(x, w, b, zz, groups=G, checkpoint=True, **kw)
        src = (kx, kz) if ckpt else (x, zz)
        g = ssd.group_norm_silu_backward(d, src[0], w, b, src[1], groups=G, **kw)
        torch.cuda.synchronize()
        return [t for t in (out, g["dx"], g["dz"], g["dweight"], g["dbias"]) if t is not None]

    forms = (dict(), dict(center=True), dict(norm_before_gate=True, center=True), dict(none=True),
             dict(none=True, center=True))
    clean = [both(**dict(f)) for f in forms]
    # (from checkpoints the whole first block reads as NaN: it is all the first group's)
    assert not ckpt or gs >= 32
    for t in (x, d):
        t[1, 0], t[2, 0], t[3, 0] = float("nan"), float("inf"), -float("inf")
    z[1, 1] = float("nan")
    w[0], b[0] = float("inf"), float("nan")
    for f, want in zip(forms, clean):
        for got, ref in zip(both(**dict(f)), want):
            assert torch.equal(got[..., gs:], ref[..., gs:]), f


def test_norm_sums_of_many_rows():
    """dweight and dbias over 200,000 tokens of few channels: each walker adds
    at most 256 rows in fp32, the walkers in fp64."""
    T, C = 200000, 64
    g = torch.Generator("cuda").manual_seed(1)
    x, z, d = (torch.randn(T, C, device="cuda", generator=g) for _ in range(3))
    w, b = torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")
    print("[gpu] group norm sums of many rows", flush=True)
    got = ssd.group_norm_silu_backward(d, x, w, b, z, groups=2)
    torch.cuda.synchronize()
    want, size = norm_backward(d.cpu(), x.cpu(), z.cpu(), w.cpu(), b.cpu(), 2, 1e-5, False, "first")
    for k in ("dx", "dz", "dweight", "dbias"):
        check(k, got[k], want[k], size[k], "fp32", 512)


def _partial_rows(T, C, G, dtype):
    """Rows of partial sums of the backward pass (the most of both sources)."""
    p = ssd.NormProblem(C, C, C, C, C, T, C, G,
                        ssd.SSD_DTYPE_BF16 if dtype == "bf16" else ssd.SSD_DTYPE_F32, 0, 1e-5)
    n = ctypes.c_size_t(0)
    assert ssd.load().ssd_group_norm_silu_backward_workspace_size(p, ctypes.byref(n)) == ssd.SSD_OK
    return n.value // (8 * C)


@pytest.mark.parametrize("T,gs,dtype,gate,center,affine", [
    # one part a lane
    (205, 1040, "bf16", "first", False, "wb"), (205, 1040, "fp32", "last", True, "wb"),
    # three (forward, and backward from 8 bits; backward from tensors two), the last nearly empty
    (67, 4104, "bf16", "last", True, "wb"), (67, 4104, "bf16", "none", False, "w"),
    (67, 4104, "fp32", "first", False, "wb"), (67, 4104, "fp32", "last", True, "wb"),
    (67, 4104, "fp32", "none", True, "wb"),
    (67, 5120, "bf16", "first", True, "wb"), (67, 5120, "bf16", "last", False, "w"),
    (67, 5120, "bf16", "none", True, "wb"), (67, 5120, "fp32", "first", False, "w"),
    (67, 5120, "fp32", "last", True, "wb"), (67, 5120, "fp32", "none", False, "wb"),
    # four forward, two backward
    (67, 8192, "bf16", "first", False, "wb"), (67, 8192, "fp32", "last", True, "wb"),
    # four
    (67, 16384, "bf16", "last", True, "wb"), (67, 16384, "fp32", "first", False, "wb"),
    (67, 16384, "fp32", "none", True, "w"),
])
def test_norm_workgroups_walk_several_rows(T, gs, dtype, gate, center, affine):
    """Groups wider than a wave, of which every workgroup takes several rows in
    turn and some one row fewer: the next row's loads, the sums' buffers taken
    in turn and the gradients summed over rows. 16 groups, of which the first
    and the last are compared with the oracle; dout holds whole numbers, so
    that dbias (gate first) is exact whatever the order of its sum. At most 8
    rows a lane: the bounds of layer_helpers hold as they are."""
    G = 16
    C = G * gs
    rng = np.random.default_rng(T + gs)
    x, xn = rows(rng, T, C, dtype)
    z, zn = rows(rng, T, C, dtype, spread=0.0) if gate != "none" else (None, None)
    dn = rng.integers(-8, 9, (T, C)).astype(np.float64)
    d = torch.from_numpy(dn).to(DT[dtype]).cuda()
    w = (1 + 0.2 * rng.standard_normal(C)).astype(np.float32) if "w" in affine else None
    b = (0.2 * rng.standard_normal(C)).astype(np.float32) if "b" in affine else None
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()
    kw = dict(groups=G, eps=1e-5, center=center, norm_before_gate=gate == "last")
    print("[gpu] group norm rows in turn %d x 16 x %d %s %s" % (T, gs, dtype, gate), flush=True)
    assert T > 2 * _partial_rows(T, C, G, dtype)
    out = ssd.group_norm_silu(x, dev(w), dev(b), z, **kw)
    same, kx, kz = ssd.group_norm_silu(x, dev(w), dev(b), z, checkpoint=True, **kw)
    plain = ssd.group_norm_silu_backward(d, x, dev(w), dev(b), z, **kw)
    kept_ = ssd.group_norm_silu_backward(d, kx, dev(w), dev(b), kz, **kw)
    torch.cuda.synchronize()
    assert torch.equal(out, same)
    for k, t in ((kx, x), (kz, z)):
        if t is not None:
            ref = ssd.checkpoint_save(t)
            assert torch.equal(k.q, ref.q) and torch.equal(k.exponents, ref.exponents)
    if gate == "first" and b is not None:
        for g in (plain, kept_):
            assert np.array_equal(g["dbias"].cpu().numpy(), dn.sum(axis=0))
    xk = kx.load().double().cpu().numpy()
    zk = None if z is None else kz.load().double().cpu().numpy()
    for at in (slice(0, gs), slice(C - gs, C)):
        cut = lambda a: None if a is None else a[..., at]
        want, size = norm(cut(xn), cut(zn), cut(w), cut(b), 1, 1e-5, center, gate)
        check("out", out[:, at], want, size, dtype, 160)
        for g, xv, zv in ((plain, xn, zn), (kept_, xk, zk)):
            want, size = norm_backward(cut(dn), cut(xv), cut(zv), cut(w), cut(b), 1, 1e-5, center,
                                       gate)
            for k in ("dx", "dz", "dweight", "dbias"):
                if g[k] is not None:
                    check(k, g[k][..., at], want[k], size[k],
                          "fp32" if k in ("dweight", "dbias") else dtype, 512)


def test_norm_sums_of_rows_side_by_side():
    """One group of 8 channels: a workgroup takes 256 rows side by side, whose
    shares of dweight and dbias are joined in fp32 before the partial rows are
    written. A lane's own 9 rows and 255 joins in turn: C = 480 + 9 + 255 (512
    of layer_helpers counts 32 rows). dout holds whole numbers: dbias is exact."""
    T, C = (1 << 20) + 37, 8
    rng = np.random.default_rng(7)
    x, xn = rows(rng, T, C, "fp32")
    z, zn = rows(rng, T, C, "fp32", spread=0.0)
    dn = rng.integers(-8, 9, (T, C)).astype(np.float64)
    d = torch.from_numpy(dn).float().cuda()
    w, b = torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")
    print("[gpu] group norm rows side by side", flush=True)
    got = ssd.group_norm_silu_backward(d, x, w, b, z)
    torch.cuda.synchronize()
    assert -(-T // 256) > 8 * _partial_rows(T, C, 1, "fp32")
    want, size = norm_backward(dn, xn, zn, None, None, 1, 1e-5, False, "first")
    assert np.array_equal(got["dbias"].cpu().numpy(), want["dbias"])
    check("dweight", got["dweight"], want["dweight"], size["dweight"], "fp32", 480 + 9 + 255)
    for k in ("dx", "dz"):
        check(k, got[k], want[k], size[k], "fp32", 512)


def test_norm_without_tokens():
    w, b = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    print("[gpu] group norm without tokens", flush=True)
    out, kx, kz = ssd.group_norm_silu(x, w, b, x, groups=2, checkpoint=True)
    g = ssd.group_norm_silu_backward(x, x, w, b, x, groups=2)
    torch.cuda.synchronize()
    assert out.shape == x.shape and kx.shape == x.shape and kz.shape == x.shape
    assert torch.count_nonzero(g["dweight"]) == 0 and torch.count_nonzero(g["dbias"]) == 0


@pytest.mark.parametrize("ckpt", [False, True])
def test_norm_writes_only_its_columns(ckpt):
    """Outputs that are slices of wider rows: the columns beside them stay."""
    T, C = 70, 640
    rng = np.random.default_rng(8)
    x, _ = rows(rng, T, C, "bf16", lead=16, pad=40)
    z, _ = rows(rng, T, C, "bf16", lead=8, pad=8)
    d, _ = rows(rng, T, C, "bf16", lead=24)
    w = torch.ones(C, device="cuda")
    wide = [torch.full((T, C + 48), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    out, dx, dz = (v[:, 16:16 + C] for v in wide)
    print("[gpu] group norm into slices", flush=True)
    want, kx, kz = ssd.group_norm_silu(x, w, None, z, checkpoint=True)
    ssd.group_norm_silu(x, w, None, z, out=out)
    src = (kx, kz) if ckpt else (x, z)
    wg = ssd.group_norm_silu_backward(d, src[0], w, None, src[1])
    g = ssd.group_norm_silu_backward(d, src[0], w, None, src[1], dx=dx, dz=dz)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and g["dx"] is dx
    assert torch.equal(dx, wg["dx"]) and torch.equal(dz, wg["dz"])
    assert torch.equal(g["dweight"], wg["dweight"])
    for v in wide:
        assert (v[:, :16] == 7).all() and (v[:, 16 + C:] == 7).all()


def test_norm_layouts():
    """3-D inputs, rows that must be copied (odd strides, transposed), expanded
    rows: all give what contiguous copies give."""
    print("[gpu] group norm layouts", flush=True)
    base = torch.randn(2, 9, 3, 64, device="cuda").to(torch.bfloat16)
    z = torch.randn(2, 9, 64, device="cuda").to(torch.bfloat16)
    for x in (base[:, :, 1], base[:, :, 1].transpose(0, 1).contiguous().transpose(0, 1),
              torch.randn(2, 9, 67, device="cuda").to(torch.bfloat16)[..., 3:],
              torch.randn(1, 1, 64, device="cuda").to(torch.bfloat16).expand(2, 9, 64)):
        got = ssd.group_norm_silu(x, None, None, z, groups=4)
        want = ssd.group_norm_silu(x.contiguous().clone(), None, None, z, groups=4)
        assert got.shape == x.shape and torch.equal(got, want)
    with pytest.raises(ValueError, match="out"):
        ssd.group_norm_silu(z, out=torch.empty(9, 2, 64, device="cuda",
                                               dtype=torch.bfloat16).transpose(0, 1))


def test_norm_past_32_bit_offsets():
    """Rows whose element offsets pass 2^32: the last rows equal a small call's."""
    T, C, pad = 33000, 1024, (1 << 17) - 1024       # 33000 * 2^17 > 2^32 elements
    print("[gpu] group norm past 32-bit offsets", flush=True)
    wide = torch.zeros(T, C + pad, dtype=torch.bfloat16, device="cuda")
    x = wide[:, :C]
    x.copy_(torch.randn(T, C, device="cuda"))
    out = torch.zeros(T, C + pad, dtype=torch.bfloat16, device="cuda")[:, pad:]
    z = torch.randn(T, C, device="cuda").to(torch.bfloat16)
    ssd.group_norm_silu(x, None, None, z, groups=2, out=out)
    g = ssd.group_norm_silu_backward(x, x, None, None, z, groups=2, dx=out)
    want = ssd.group_norm_silu_backward(x[-5:].clone(), x[-5:].clone(), None, None, z[-5:],
                                        groups=2)
    torch.cuda.synchronize()
    assert torch.equal(out[-5:], want["dx"]) and torch.equal(g["dz"][-5:], want["dz"])


def test_norm_on_another_stream_and_twice():
    """A call on a side stream, and the same call again: equal bits."""
    t, _ = _inputs("rows-2.7b")
    print("[gpu] group norm on a side stream", flush=True)
    want = ssd.group_norm_silu(t["x"], t["w"], t["b"], t["z"], **t["kw"])
    wg = ssd.group_norm_silu_backward(t["d"], t["x"], t["w"], t["b"], t["z"], **t["kw"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = ssd.group_norm_silu(t["x"], t["w"], t["b"], t["z"], stream=s, **t["kw"])
    g = ssd.group_norm_silu_backward(t["d"], t["x"], t["w"], t["b"], t["z"], stream=s, **t["kw"])
    s.synchronize()
    assert torch.equal(out, want)
    for k in ("dx", "dz", "dweight"):
        assert torch.equal(g[k], wg[k]), k
