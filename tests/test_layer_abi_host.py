"""The C ABI of the operators around the SSD layer on the host (argument
checks and workspace sizes; nothing is launched), and the Python binding's
refusals on torch's "meta" device."""
import ctypes

import pytest
import torch

import mamba_ssd_sequence_fwd_amd as ssd
from mamba_ssd_sequence_fwd_amd import _lib

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    return ssd.load()


def _addr(i):
    return vp(4096 * (i + 1))


def CK(q=1 << 20, e=1 << 21):
    return _lib.CheckpointArg(q, e)


# ---- group norm ------------------------------------------------------------------


def NP(**kw):
    base = dict(x_stride=96, z_stride=96, out_stride=96, dx_stride=96, dz_stride=96, tokens=10,
                channels=96, groups=2, dtype=ssd.SSD_DTYPE_BF16, flags=0, eps=1e-5)
    base.update(kw)
    return _lib.NormProblem(**base)


def _norm(lib, prob, x=0, z=1, out=4, kx=None, kz=None):
    p = lambda i: None if i is None else i if isinstance(i, vp) else _addr(i)
    return lib.ssd_group_norm_silu(None if prob is None else ctypes.byref(prob), p(x), p(z),
                                   _addr(2), _addr(3), p(out), kx, kz, None)


NORM_BAD = [
    ({"tokens": -1}, ssd.SSD_ERR_INVALID_ARG),
    ({"channels": 0}, ssd.SSD_ERR_INVALID_ARG),
    ({"groups": 0}, ssd.SSD_ERR_INVALID_ARG),
    ({"groups": 5}, ssd.SSD_ERR_INVALID_ARG),
    ({"flags": 4}, ssd.SSD_ERR_INVALID_ARG),
    ({"eps": -1e-5}, ssd.SSD_ERR_INVALID_ARG),
    ({"eps": float("nan")}, ssd.SSD_ERR_INVALID_ARG),
    ({"eps": float("inf")}, ssd.SSD_ERR_INVALID_ARG),
    ({"dtype": 3}, ssd.SSD_ERR_UNSUPPORTED),
    ({"groups": 24}, ssd.SSD_ERR_UNSUPPORTED),                       # 4 channels a group
    ({"tokens": 1 << 30}, ssd.SSD_ERR_UNSUPPORTED),
    ({"channels": 16392, "groups": 1, "x_stride": 16392, "z_stride": 16392,
      "out_stride": 16392, "dx_stride": 16392, "dz_stride": 16392}, ssd.SSD_ERR_UNSUPPORTED),
    ({"x_stride": 88}, ssd.SSD_ERR_INVALID_ARG),
    ({"z_stride": 100}, ssd.SSD_ERR_INVALID_ARG),                    # 200 bytes
    ({"out_stride": 1 << 33}, ssd.SSD_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", NORM_BAD)
def test_norm_refuses(lib, kw, status):
    assert _norm(lib, NP(**kw)) == status


def test_norm_refuses_pointers(lib):
    assert _norm(lib, None) == ssd.SSD_ERR_INVALID_ARG
    assert _norm(lib, NP(), x=None) == ssd.SSD_ERR_INVALID_ARG
    assert _norm(lib, NP(), out=None) == ssd.SSD_ERR_INVALID_ARG
    for k in ("x", "z", "out"):
        assert _norm(lib, NP(), **{k: vp(4096 + 8)}) == ssd.SSD_ERR_INVALID_ARG
    # the gate's place needs a gate
    assert _norm(lib, NP(flags=ssd.SSD_NORM_BEFORE_GATE), z=None) == ssd.SSD_ERR_INVALID_ARG
    # checkpoints of both or neither, complete and aligned
    assert _norm(lib, NP(), kx=CK()) == ssd.SSD_ERR_INVALID_ARG
    assert _norm(lib, NP(), kz=CK()) == ssd.SSD_ERR_INVALID_ARG
    assert _norm(lib, NP(), z=None, kx=CK(), kz=CK()) == ssd.SSD_ERR_INVALID_ARG
    assert _norm(lib, NP(), kx=CK(q=None), kz=CK()) == ssd.SSD_ERR_INVALID_ARG
    assert _norm(lib, NP(), kx=CK(), kz=CK(e=None)) == ssd.SSD_ERR_INVALID_ARG
    assert _norm(lib, NP(), kx=CK(q=(1 << 20) + 4), kz=CK()) == ssd.SSD_ERR_INVALID_ARG
    assert b"8-byte" in lib.ssd_last_error_detail()


def test_norm_without_tokens_is_a_no_op(lib):
    assert _norm(lib, NP(tokens=0), x=None, z=None, out=None) == ssd.SSD_OK


def _norm_back(lib, prob, dout=0, x=1, z=2, kx=None, kz=None, dx=5, dz=6, dw=7, db=8, ws=9,
               wsb=1 << 30):
    p = lambda i: None if i is None else i if isinstance(i, vp) else _addr(i)
    return lib.ssd_group_norm_silu_backward(
        None if prob is None else ctypes.byref(prob), p(dout), p(x), p(z), kx, kz, _addr(3),
        _addr(4), p(dx), p(dz), p(dw), p(db), p(ws), ctypes.c_size_t(wsb), None)


@pytest.mark.parametrize("kw,status", NORM_BAD + [
    ({"dx_stride": 8}, ssd.SSD_ERR_INVALID_ARG),
    ({"dz_stride": 97}, ssd.SSD_ERR_INVALID_ARG),
])
def test_norm_backward_refuses(lib, kw, status):
    assert _norm_back(lib, NP(**kw)) == status


def test_norm_backward_refuses_pointers(lib):
    bad = ssd.SSD_ERR_INVALID_ARG
    for k in ("dout", "dx", "dz"):
        assert _norm_back(lib, NP(), **{k: None}) == bad, k
        assert _norm_back(lib, NP(), **{k: vp(4096 + 8)}) == bad, k
    assert _norm_back(lib, NP(), x=None, z=None) == bad
    assert _norm_back(lib, NP(), kx=CK(), kz=CK()) == bad              # both forms
    assert _norm_back(lib, NP(), x=None, kx=CK()) == bad               # one of each
    assert _norm_back(lib, NP(), z=None, kz=CK()) == bad
    assert _norm_back(lib, NP(), x=None, z=None, kx=CK(), kz=CK(q=None)) == bad
    assert _norm_back(lib, NP(flags=2), z=None) == bad
    assert _norm_back(lib, NP(), ws=None) == ssd.SSD_ERR_WORKSPACE
    assert _norm_back(lib, NP(), ws=vp(4096 + 128)) == ssd.SSD_ERR_WORKSPACE
    n = ctypes.c_size_t(0)
    assert lib.ssd_group_norm_silu_backward_workspace_size(ctypes.byref(NP()),
                                                           ctypes.byref(n)) == ssd.SSD_OK
    assert n.value >= 2 * 96 * 4 and n.value % (2 * 96 * 4) == 0
    assert _norm_back(lib, NP(), wsb=n.value - 1) == ssd.SSD_ERR_WORKSPACE
    assert lib.ssd_group_norm_silu_backward_workspace_size(ctypes.byref(NP()), None) == bad


def test_norm_backward_workspace_is_small(lib):
    """At most 2048 partial rows of 8 bytes a channel, or one for 256 tokens
    where that is more."""
    n = ctypes.c_size_t(0)
    for channels, groups in ((5120, 1), (4096, 8), (64, 8), (8, 1)):
        for tokens in (1, 100, 1 << 14, 1 << 23):
            p = NP(tokens=tokens, channels=channels, groups=groups)
            assert lib.ssd_group_norm_silu_backward_workspace_size(
                ctypes.byref(p), ctypes.byref(n)) == ssd.SSD_OK
            assert 0 < n.value <= max(2048, -(-tokens // 256)) * 8 * channels


# ---- convolution front -------------------------------------------------------------


def CP(**kw):
    base = dict(batch=2, seqlen=100, num_seqs=0, x_dim=64, bc_dim=16, width=4, in_stride=96,
                dtype=ssd.SSD_DTYPE_BF16, flags=0)
    base.update(kw)
    return ssd.ConvProblem(**base)


def _conv_ck(lib, prob, xbc=0, ck=None, hist_out=8, cu=None):
    p = lambda i: None if i is None else _addr(i)
    return lib.ssd_conv1d_silu_checkpoint(ctypes.byref(prob), p(xbc), ck, _addr(1), _addr(2),
                                          _addr(3), p(cu), _addr(5), _addr(6), _addr(7),
                                          p(hist_out), None)


def test_conv_checkpoint_refuses(lib):
    bad = ssd.SSD_ERR_INVALID_ARG
    assert _conv_ck(lib, CP()) == bad                                   # no checkpoint
    assert _conv_ck(lib, CP(), ck=CK(q=None)) == bad
    assert _conv_ck(lib, CP(), ck=CK(q=(1 << 20) + 2)) == bad
    assert _conv_ck(lib, CP(), xbc=None, ck=CK()) == bad                # exact history
    assert b"history" in lib.ssd_last_error_detail()
    assert _conv_ck(lib, CP(width=5), ck=CK()) == ssd.SSD_ERR_UNSUPPORTED
    assert _conv_ck(lib, CP(batch=1, num_seqs=2), ck=CK()) == bad       # no offsets
    assert _conv_ck(lib, CP(batch=0), ck=CK()) == ssd.SSD_OK


def test_conv_without_tokens_keeps_its_history(lib):
    """No tokens: xbc is an empty tensor's NULL, which does not stand for a
    recomputation, so history_out is allowed (no sequences: nothing is launched)."""
    for ck in (CK(), CK(q=None, e=None)):
        assert _conv_ck(lib, CP(batch=0), xbc=None, ck=ck) == ssd.SSD_OK
        assert _conv_ck(lib, CP(), xbc=None, ck=CK()) == ssd.SSD_ERR_INVALID_ARG


def _conv_back(lib, prob, ck=None, cu=None, stride=96, wsb=1 << 40, **over):
    names = ["xbc", "weight", "bias", "hist", "dx", "dB", "dC", "dho", "dxbc", "dw", "db", "dh",
             "ws"]
    a = {n: _addr(i) for i, n in enumerate(names)}
    a.update(over)
    return lib.ssd_conv1d_silu_backward(
        ctypes.byref(prob), a["xbc"], ck, a["weight"], a["bias"], a["hist"], cu, a["dx"], a["dB"],
        a["dC"], a["dho"], a["dxbc"], stride, a["dw"], a["db"], a["dh"], a["ws"],
        ctypes.c_size_t(wsb), None)


@pytest.mark.parametrize("kw,status", [
    ({"batch": -1}, ssd.SSD_ERR_INVALID_ARG),
    ({"seqlen": -1}, ssd.SSD_ERR_INVALID_ARG),
    ({"flags": 1}, ssd.SSD_ERR_INVALID_ARG),
    ({"in_stride": 88}, ssd.SSD_ERR_INVALID_ARG),
    ({"in_stride": 100}, ssd.SSD_ERR_INVALID_ARG),
    ({"num_seqs": 3}, ssd.SSD_ERR_INVALID_ARG),
    ({"batch": 1, "num_seqs": 3}, ssd.SSD_ERR_INVALID_ARG),            # no offsets
    ({"dtype": 5}, ssd.SSD_ERR_UNSUPPORTED),
    ({"width": 1}, ssd.SSD_ERR_UNSUPPORTED),
    ({"x_dim": 60}, ssd.SSD_ERR_UNSUPPORTED),
    ({"seqlen": 1 << 29, "batch": 2}, ssd.SSD_ERR_UNSUPPORTED),
])
def test_conv_backward_refuses(lib, kw, status):
    assert _conv_back(lib, CP(**kw)) == status


def test_conv_backward_refuses_pointers(lib):
    bad = ssd.SSD_ERR_INVALID_ARG
    for k in ("xbc", "weight", "dx", "dB", "dC", "dxbc", "dw"):
        assert _conv_back(lib, CP(), **{k: None}) == bad, k
    for k in ("xbc", "hist", "dx", "dB", "dC", "dho", "dxbc", "dh"):
        assert _conv_back(lib, CP(), **{k: vp((1 << 16) + 8)}) == bad, k
    assert _conv_back(lib, CP(), ck=CK()) == bad                        # both forms
    assert _conv_back(lib, CP(), xbc=None, ck=CK(e=None)) == bad
    assert _conv_back(lib, CP(), stride=88) == bad
    assert _conv_back(lib, CP(), stride=100) == bad
    assert _conv_back(lib, CP(), ws=None) == ssd.SSD_ERR_WORKSPACE
    n = ctypes.c_size_t(0)
    assert lib.ssd_conv1d_silu_backward_workspace_size(ctypes.byref(CP()),
                                                       ctypes.byref(n)) == ssd.SSD_OK
    assert n.value > 0 and n.value % (5 * 96 * 4) == 0
    assert _conv_back(lib, CP(), wsb=n.value - 1) == ssd.SSD_ERR_WORKSPACE
    packed = CP(batch=1, num_seqs=7)
    assert lib.ssd_conv1d_silu_backward_workspace_size(ctypes.byref(packed),
                                                       ctypes.byref(n)) == ssd.SSD_OK
    assert lib.ssd_conv1d_silu_backward_workspace_size(ctypes.byref(packed), None) == bad


@pytest.mark.parametrize("in_stride", [0, 88, 100])
def test_conv_from_a_checkpoint_needs_no_input_stride(lib, in_stride):
    """in_stride belongs to xbc: looked at where xbc is given, and only there.
    (No sequences or no workspace: the calls end before a launch.)"""
    n, want = ctypes.c_size_t(0), ctypes.c_size_t(0)
    size = lib.ssd_conv1d_silu_backward_workspace_size
    assert size(ctypes.byref(CP()), ctypes.byref(want)) == ssd.SSD_OK
    assert size(ctypes.byref(CP(in_stride=in_stride)), ctypes.byref(n)) == ssd.SSD_OK
    assert n.value == want.value
    p, none = CP(in_stride=in_stride), CP(batch=0, in_stride=in_stride)
    assert _conv_ck(lib, none, xbc=None, ck=CK(), hist_out=None) == ssd.SSD_OK
    assert _conv_back(lib, p, xbc=None, ck=CK(), ws=None) == ssd.SSD_ERR_WORKSPACE
    bad = ssd.SSD_ERR_INVALID_ARG
    assert _conv_ck(lib, p, ck=CK()) == bad
    assert _conv_ck(lib, none, ck=CK()) == bad
    assert _conv_back(lib, p) == bad
    assert b"in_stride" in lib.ssd_last_error_detail()


# ---- checkpoints -------------------------------------------------------------------


def KP(**kw):
    base = dict(rows=10, stride=48, channels=40, dtype=ssd.SSD_DTYPE_BF16, flags=0)
    base.update(kw)
    return _lib.CheckpointProblem(**base)


@pytest.mark.parametrize("fn", ["ssd_checkpoint_save", "ssd_checkpoint_load"])
def test_checkpoint_refuses(lib, fn):
    def call(prob, tensor=_addr(0), ck=CK()):
        args = (tensor, ck) if fn.endswith("save") else (ck, tensor)
        return getattr(lib, fn)(None if prob is None else ctypes.byref(prob), *args, None)

    bad = ssd.SSD_ERR_INVALID_ARG
    assert call(None) == bad
    for kw, status in (({"rows": -1}, bad), ({"channels": 0}, bad), ({"flags": 1}, bad),
                       ({"stride": 32}, bad), ({"stride": 44}, bad), ({"stride": 1 << 32}, bad),
                       ({"dtype": 2}, ssd.SSD_ERR_UNSUPPORTED),
                       ({"channels": 36}, ssd.SSD_ERR_UNSUPPORTED),
                       ({"rows": 1 << 31}, ssd.SSD_ERR_UNSUPPORTED)):
        assert call(KP(**kw)) == status, kw
    assert call(KP(), tensor=None) == bad
    assert call(KP(), tensor=vp(4096 + 8)) == bad
    assert call(KP(), ck=None) == bad
    assert call(KP(), ck=CK(q=None)) == bad
    assert call(KP(), ck=CK(q=(1 << 20) + 1)) == bad
    assert call(KP(rows=0), tensor=None, ck=None) == ssd.SSD_OK


# ---- the Python binding -------------------------------------------------------------


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_checkpoint_checks_its_parts():
    q, e = torch.zeros(3, 40, dtype=torch.int8), torch.zeros(3, 2, dtype=torch.uint8)
    k = ssd.Checkpoint(q, e, torch.bfloat16)
    assert k.shape == (3, 40) and k.nbytes == 126 and k.device.type == "cpu"
    for bad in ((q.float(), e, torch.bfloat16), (q, e.int(), torch.bfloat16),
                (q, e, torch.float16), (q[:, :36], e, torch.bfloat16),
                (torch.zeros(3, 36, dtype=torch.int8), e, torch.bfloat16),
                (q, e[:, :1], torch.bfloat16), (q, e.t(), torch.bfloat16)):
        with pytest.raises(ValueError):
            ssd.Checkpoint(*bad)
    with pytest.raises(ValueError, match="GPU"):
        k.load()
    with pytest.raises(ValueError, match="GPU"):
        ssd.checkpoint_save(torch.zeros(3, 40))


@pytest.mark.parametrize("name", ["weight", "bias", "z", "out"])
def test_norm_rejects_tensor_on_another_device(name):
    a = dict(weight=_meta(64, dtype=torch.float32), bias=_meta(64, dtype=torch.float32),
             z=_meta(5, 64), out=_meta(5, 64))
    a[name] = torch.zeros(a[name].shape, dtype=a[name].dtype)
    with pytest.raises(ValueError, match=name):
        ssd.group_norm_silu(_meta(5, 64), **a)
    with pytest.raises(ValueError, match="GPU"):
        ssd.group_norm_silu(_meta(5, 64))


@pytest.mark.parametrize("name", ["dout", "weight", "bias", "dx", "dz"])
def test_norm_backward_rejects_tensor_on_another_device(name):
    a = dict(dout=_meta(5, 64), weight=_meta(64, dtype=torch.float32),
             bias=_meta(64, dtype=torch.float32), dx=_meta(5, 64), dz=_meta(5, 64))
    a[name] = torch.zeros(a[name].shape, dtype=a[name].dtype)
    with pytest.raises(ValueError, match=name):
        ssd.group_norm_silu_backward(x=_meta(5, 64), z=_meta(5, 64), **a)


def test_norm_backward_takes_tensors_or_checkpoints():
    k = ssd.Checkpoint(torch.zeros(5, 64, dtype=torch.int8), torch.zeros(5, 2, dtype=torch.uint8),
                       torch.bfloat16)
    t = torch.zeros(5, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="both"):
        ssd.group_norm_silu_backward(t, k, z=t)
    with pytest.raises(ValueError, match="both"):
        ssd.group_norm_silu_backward(t, t, z=k)


@pytest.mark.parametrize("name", ["weight", "bias", "dx", "dB", "dC", "history", "dhistory_out",
                                  "dxbc"])
def test_conv_backward_rejects_tensor_on_another_device(name):
    ch = 64 + 2 * 16
    a = dict(weight=_meta(ch, 4, dtype=torch.float32), bias=_meta(ch, dtype=torch.float32),
             dx=_meta(2, 32, 64), dB=_meta(2, 32, 16), dC=_meta(2, 32, 16),
             history=_meta(2, 3, ch), dhistory_out=_meta(2, 3, ch), dxbc=_meta(2, 32, ch))
    a[name] = torch.zeros(a[name].shape, dtype=a[name].dtype)
    with pytest.raises(ValueError, match=name):
        ssd.conv1d_silu_backward(_meta(2, 32, ch), **a)


def test_conv_refuses_a_checkpoint_of_a_checkpoint():
    k = ssd.Checkpoint(torch.zeros(2, 5, 96, dtype=torch.int8),
                       torch.zeros(2, 5, 3, dtype=torch.uint8), torch.bfloat16)
    w = torch.zeros(96, 4)
    with pytest.raises(ValueError, match="already"):
        ssd.conv1d_silu(k, w, None, 64, 16, checkpoint=True)
    with pytest.raises(ValueError, match="history_out"):
        ssd.conv1d_silu(k, w, None, 64, 16, history_out=torch.zeros(2, 3, 96))


def test_binding_refuses_sizes_that_would_wrap():
    """Sizes past 32 bits are refused before they are put into a C structure."""
    far = _meta(2 ** 32 + 5, 8)
    with pytest.raises(ValueError, match="tokens"):
        ssd.group_norm_silu(far)
    with pytest.raises(ValueError, match="tokens"):
        ssd.group_norm_silu_backward(far, far)
    with pytest.raises(ValueError, match="groups"):
        ssd.group_norm_silu(_meta(4, 64), groups=2 ** 32 + 1)
    for groups in (0, -1, 65):
        with pytest.raises(ValueError, match="groups"):
            ssd.group_norm_silu(_meta(4, 64), groups=groups)


def test_front_refuses_sizes_past_32_bits(monkeypatch):
    # sizes that the C structure's 32 bits would wrap to small valid ones
    monkeypatch.setattr(_lib, "_on_gpu", lambda dev: None)
    w, many = _meta(8, 4, dtype=torch.float32), (1 << 32) + 8
    kept = ssd.Checkpoint(_meta(1, many, 8, dtype=torch.int8),
                          _meta(1, many, 1, dtype=torch.uint8), torch.bfloat16)
    for xbc in (_meta(1, many, 8), _meta(1 << 20, 1 << 12, 8), kept):
        with pytest.raises(ValueError, match="more than one call takes"):
            ssd.conv1d_silu(xbc, w, None, 8, 0)
    far = torch.empty_strided((1, 2, 8), (1 << 33, 1 << 32, 1), dtype=torch.bfloat16,
                              device="meta")
    with pytest.raises(ValueError, match="more than one call takes"):
        ssd.conv1d_silu(far, w, None, 8, 0)


def test_norm_refuses_what_is_not_a_pair_to_fill(monkeypatch):
    monkeypatch.setattr(_lib, "_on_gpu", lambda dev: None)
    monkeypatch.setattr(_lib, "_stream_of", lambda dev, stream: (_lib._NO_CONTEXT, None))
    x, z = _meta(5, 64), _meta(5, 64)
    one = ssd.Checkpoint(_meta(5, 64, dtype=torch.int8), _meta(5, 2, dtype=torch.uint8), x.dtype)
    for given in (one, (one,), (one, one), (one, one, one)):
        with pytest.raises(ValueError, match="pair|each"):
            ssd.group_norm_silu(x, z=z, checkpoint=given)
    with pytest.raises(ValueError, match="True, False or a Checkpoint"):
        ssd.group_norm_silu(x, z=z, checkpoint=(one, None))


def test_refuses_what_no_launch_holds(lib):
    """Sizes whose grids would pass 2^32 threads are refused before a launch."""
    n = ctypes.c_size_t(0)
    no = ssd.SSD_ERR_UNSUPPORTED
    many = CP(batch=1, seqlen=(1 << 30) - 8, x_dim=8, bc_dim=0, in_stride=8)
    assert lib.ssd_conv1d_silu_backward_workspace_size(ctypes.byref(many), ctypes.byref(n)) == no
    assert _conv_ck(lib, many, ck=CK(), hist_out=None) == no
    wide = CP(batch=1, seqlen=1, x_dim=1 << 26, bc_dim=0, in_stride=1 << 26)
    assert lib.ssd_conv1d_silu_backward_workspace_size(ctypes.byref(wide), ctypes.byref(n)) == no
    c = 1 << 27
    p = NP(tokens=1, channels=c, groups=c // 64, **{k + "_stride": c for k in
                                                    ("x", "z", "out", "dx", "dz")})
    assert _norm(lib, p) == no
    for fn in (lib.ssd_checkpoint_save, lib.ssd_checkpoint_load):
        prob, ck = KP(rows=1 << 30, channels=256, stride=256), CK()
        a = (_addr(0), ctypes.byref(ck)) if fn is lib.ssd_checkpoint_save else \
            (ctypes.byref(ck), _addr(0))
        assert fn(ctypes.byref(prob), *a, None) == no


def test_a_checkpoint_where_a_tensor_belongs_is_refused(monkeypatch):
    """A Checkpoint has a tensor's shape, dtype and device: refused by name, not
    by a missing attribute."""
    monkeypatch.setattr(_lib, "_on_gpu", lambda dev: None)

    def K(*shape, dtype=torch.bfloat16):
        return ssd.Checkpoint(_meta(*shape, dtype=torch.int8),
                              _meta(*shape[:-1], -(-shape[-1] // 32), dtype=torch.uint8), dtype)

    def refused(name, call, *a, **kw):
        with pytest.raises(ValueError, match="^%s is a Checkpoint" % name):
            call(*a, **kw)

    t, f = _meta(5, 64), torch.float32
    refused("x", ssd.group_norm_silu, K(5, 64))
    refused("z", ssd.group_norm_silu, t, z=K(5, 64))
    refused("out", ssd.group_norm_silu, t, out=K(5, 64))
    refused("weight", ssd.group_norm_silu, t, K(64, dtype=f))
    refused("bias", ssd.group_norm_silu, t, None, K(64, dtype=f))
    back = ssd.group_norm_silu_backward
    for x in (t, K(5, 64)):
        refused("dout", back, K(5, 64), x)
        refused("dx", back, t, x, dx=K(5, 64))
        refused("dz", back, t, x, z=x, dz=K(5, 64))
    away = ssd.Checkpoint(torch.zeros(5, 64, dtype=torch.int8),
                          torch.zeros(5, 2, dtype=torch.uint8), torch.bfloat16)
    with pytest.raises(ValueError, match="z is on cpu"):
        back(t, K(5, 64), z=away)
    refused("tensor", ssd.checkpoint_save, K(5, 64))
    refused("out", K(5, 64).load, out=K(5, 64))
    ch = 64 + 2 * 16
    w, b = _meta(ch, 4, dtype=f), _meta(ch, dtype=f)
    for xbc in (_meta(2, 32, ch), K(2, 32, ch)):
        refused("history", ssd.conv1d_silu, xbc, w, b, 64, 16, K(2, 3, ch))
        for name, n in (("x", 64), ("B", 16), ("C", 16)):
            refused(name, ssd.conv1d_silu, xbc, w, b, 64, 16, **{name: K(2, 32, n)})
        for name, k in (("dx", K(2, 32, 64)), ("dB", K(2, 32, 16)), ("dC", K(2, 32, 16)),
                        ("history", K(2, 3, ch)), ("dhistory_out", K(2, 3, ch)),
                        ("dxbc", K(2, 32, ch)), ("weight", K(ch, 8, dtype=f)),
                        ("bias", K(ch, dtype=f))):
            a = dict(weight=w, bias=b, dx=_meta(2, 32, 64), dB=_meta(2, 32, 16),
                     dC=_meta(2, 32, 16))
            a[name] = k
            refused(name, ssd.conv1d_silu_backward, xbc, **a)


def test_conv_backward_takes_packed_gradients_as_the_layer_returns_them():
    """Packed: the layer's gradients have a batch axis of 1 before the tokens,
    which the packed input has not."""
    after = lambda lead, *shape: _lib._channels_after(lead, "dx", _meta(*shape), torch.bfloat16)
    for T in (1, 37):
        assert after((T,), 1, T, 4, 16) == 64 and after((T,), 1, T, 64) == 64
        assert after((T,), T, 4, 16) == 64 and after((T,), T, 64) == 64
    assert after((0,), 1, 0, 4, 16) == 64 and after((1, 37), 1, 37, 4, 16) == 64
    for lead, shape in (((37,), (2, 37, 64)), ((37,), (1, 36, 64)), ((37,), (1, 37)),
                        ((1, 37), (37, 64)), ((2, 37), (1, 2, 37, 64))):
        with pytest.raises(ValueError, match="dx must be"):
            after(lead, *shape)
