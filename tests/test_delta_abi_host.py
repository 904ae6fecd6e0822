"""The C ABI of the gated delta rule and of the norm and rotation of its keys and
queries on the host (argument checks and workspace sizes; nothing is launched),
and the Python binding's refusals on torch's "meta" device."""
import ctypes

import pytest
import torch

import mamba_ssd_sequence_fwd_amd as ssd
from mamba_ssd_sequence_fwd_amd import _lib

vp = ctypes.c_void_p
BAD, NOT_OFFERED, WS = ssd.SSD_ERR_INVALID_ARG, ssd.SSD_ERR_UNSUPPORTED, ssd.SSD_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return ssd.load()


def _addr(i):
    return vp(4096 * (i + 1))


def _p(i):
    return None if i is None else i if isinstance(i, vp) else _addr(i)


# ---- delta rule --------------------------------------------------------------------


def DP(batch=2, seqlen=100, nheads=4, headdim=64, dstate=64, ngroups=2, num_seqs=0,
       dtype=ssd.SSD_DTYPE_BF16, flags=0):
    return _lib.Problem(batch, seqlen, nheads, headdim, dstate, ngroups, 0, num_seqs, dtype, flags)


def _forward(lib, prob, x=0, g=1, beta=2, B=3, C=4, h0=5, cu=None, y=7, hT=8, ws=9, wsb=1 << 40):
    return lib.ssd_delta_forward(None if prob is None else prob, *(_p(v) for v in
                                 (x, g, beta, B, C, h0, cu, y, hT, ws)), wsb, None)


def _backward(lib, prob, x=0, g=1, beta=2, B=3, C=4, h0=5, cu=None, dy=7, dhT=8, dx=9, dg=10,
              dbeta=11, dB=12, dC=13, dh0=14, ws=15, wsb=1 << 40):
    return lib.ssd_delta_backward(None if prob is None else prob, *(_p(v) for v in (
        x, g, beta, B, C, h0, cu, dy, dhT, dx, dg, dbeta, dB, dC, dh0, ws)), wsb, None)


def _step(lib, prob, x=0, g=1, beta=2, B=3, C=4, state=5, y=6):
    return lib.ssd_delta_step(None if prob is None else prob, *(_p(v) for v in (
        x, g, beta, B, C, state, y)), None)


REFUSED = [
    (dict(batch=-1), BAD), (dict(nheads=0), BAD), (dict(headdim=0), BAD), (dict(dstate=0), BAD),
    (dict(ngroups=0), BAD), (dict(ngroups=3), BAD), (dict(flags=1), BAD),
    (dict(dtype=3), NOT_OFFERED), (dict(headdim=24), NOT_OFFERED), (dict(headdim=256), NOT_OFFERED),
    (dict(dstate=24), NOT_OFFERED), (dict(dstate=272), NOT_OFFERED),
    (dict(batch=1 << 24), NOT_OFFERED),
]
REFUSED_SEQUENCES = [
    (dict(seqlen=-1), BAD), (dict(num_seqs=-1), BAD), (dict(num_seqs=3), BAD),
    (dict(seqlen=1 << 30), NOT_OFFERED), (dict(batch=1 << 15, seqlen=1 << 15), NOT_OFFERED),
    (dict(nheads=1 << 20, ngroups=1 << 20, dstate=256), NOT_OFFERED),
    (dict(batch=1, seqlen=1 << 20, nheads=2048, headdim=128), NOT_OFFERED),
]


@pytest.mark.parametrize("kw,status", REFUSED + REFUSED_SEQUENCES)
def test_delta_refuses(lib, kw, status):
    n = ctypes.c_size_t(0)
    assert _forward(lib, DP(**kw)) == status
    assert _backward(lib, DP(**kw)) == status
    assert lib.ssd_delta_workspace_size(DP(**kw), ctypes.byref(n)) == status
    assert lib.ssd_delta_backward_workspace_size(DP(**kw), ctypes.byref(n)) == status


@pytest.mark.parametrize("kw,status", REFUSED + [(dict(seqlen=2), BAD), (dict(num_seqs=1), BAD)])
def test_delta_step_refuses(lib, kw, status):
    assert _step(lib, DP(**dict(dict(seqlen=1), **kw))) == status


def test_delta_refuses_pointers(lib):
    off = vp(4096 + 8)
    for k in ("x", "g", "beta", "B", "C", "y"):
        assert _forward(lib, DP(), **{k: None}) == BAD, k
        assert _step(lib, DP(seqlen=1), **{k: None}) == BAD, k
    for k in ("x", "B", "C", "y", "h0", "hT"):
        assert _forward(lib, DP(), **{k: off}) == BAD, k
    for k in ("x", "B", "C", "y", "state"):
        assert _step(lib, DP(seqlen=1), **{k: off}) == BAD, k
    assert _step(lib, DP(seqlen=1), state=None) == BAD
    for k in ("x", "g", "beta", "B", "C", "dy", "dx", "dg", "dbeta", "dB", "dC"):
        assert _backward(lib, DP(), **{k: None}) == BAD, k
    for k in ("x", "B", "C", "dy", "dhT", "dx", "dB", "dC", "h0", "dh0"):
        assert _backward(lib, DP(), **{k: off}) == BAD, k
    assert _forward(lib, None) == _backward(lib, None) == _step(lib, None) == BAD
    packed = DP(batch=1, num_seqs=3)
    assert _forward(lib, packed) == _backward(lib, packed) == BAD
    assert b"cu_seqlens" in lib.ssd_last_error_detail()
    assert lib.ssd_delta_workspace_size(DP(), None) == BAD
    assert lib.ssd_delta_backward_workspace_size(DP(), None) == BAD


@pytest.mark.parametrize("kw", [dict(), dict(batch=1, num_seqs=3), dict(dtype=ssd.SSD_DTYPE_F32),
                                dict(batch=1, seqlen=4096), dict(batch=1, seqlen=4096, num_seqs=2)])
def test_delta_workspace(lib, kw):
    n = ctypes.c_size_t(0)
    cu = 6 if "num_seqs" in kw else None
    for size, call, ws in ((lib.ssd_delta_workspace_size, _forward, 9),
                           (lib.ssd_delta_backward_workspace_size, _backward, 15)):
        assert size(DP(**kw), ctypes.byref(n)) == ssd.SSD_OK and n.value > 0
        assert call(lib, DP(**kw), cu=cu, ws=None) == WS
        assert call(lib, DP(**kw), cu=cu, ws=vp(4096 + 128)) == WS
        assert call(lib, DP(**kw), cu=cu, wsb=n.value - 1) == WS


def test_delta_workspace_of_long_calls(lib):
    """Bytes past 32 bits, and what grows with the tokens: the triangular matrices
    (15 KB a chunk and head in bf16) and no more than as much for the segments."""
    n = ctypes.c_size_t(0)
    p = DP(batch=1, seqlen=1 << 20, nheads=256, headdim=64, dstate=128, ngroups=1)
    assert lib.ssd_delta_workspace_size(p, ctypes.byref(n)) == ssd.SSD_OK
    chunks = (1 << 20) // 64
    assert n.value == chunks * 256 * 15 * 1024 > 1 << 32
    p = DP(batch=1, seqlen=1 << 20, nheads=16, headdim=64, dstate=128, ngroups=1)
    assert lib.ssd_delta_workspace_size(p, ctypes.byref(n)) == ssd.SSD_OK
    assert chunks * 16 * 15 * 1024 < n.value < 2 * chunks * 16 * 15 * 1024


def test_delta_without_work_is_a_no_op(lib):
    none = dict(x=None, g=None, beta=None, B=None, C=None, ws=None)
    assert _forward(lib, DP(batch=0), y=None, **none) == ssd.SSD_OK
    assert _forward(lib, DP(seqlen=0), y=None, hT=None, **none) == ssd.SSD_OK
    grads = dict(dy=None, dx=None, dg=None, dbeta=None, dB=None, dC=None)
    assert _backward(lib, DP(batch=0), **none, **grads) == ssd.SSD_OK
    assert _backward(lib, DP(seqlen=0), dh0=None, **none, **grads) == ssd.SSD_OK
    assert _step(lib, DP(batch=0, seqlen=1), x=None, state=None) == ssd.SSD_OK


# ---- norm and rotation -------------------------------------------------------------


def NP(**kw):
    base = dict(b_stride=256, c_stride=512, b_out_stride=256, c_out_stride=512, db_stride=256,
                dc_stride=512, tokens=10, b_heads=2, c_heads=4, dim=128, rotary_dim=64, period=10,
                dtype=ssd.SSD_DTYPE_BF16, flags=0, eps=1e-6)
    base.update(kw)
    return _lib.BcNormProblem(**base)


def _norm(lib, prob, B=0, C=1, bw=2, cw=3, pos=4, freqs=5, bo=6, co=7):
    return lib.ssd_bc_norm(prob, *(_p(v) for v in (B, C, bw, cw, pos, freqs, bo, co)), None)


def _norm_back(lib, prob, dbo=0, dco=1, B=2, C=3, bw=4, cw=5, pos=6, freqs=7, dB=8, dC=9, dbw=10,
               dcw=11, ws=12, wsb=1 << 40):
    return lib.ssd_bc_norm_backward(prob, *(_p(v) for v in (
        dbo, dco, B, C, bw, cw, pos, freqs, dB, dC, dbw, dcw, ws)), wsb, None)


NORM_REFUSED = [
    (dict(tokens=-1), BAD), (dict(b_heads=0), BAD), (dict(c_heads=0), BAD), (dict(dim=0), BAD),
    (dict(rotary_dim=-8), BAD), (dict(rotary_dim=12), BAD), (dict(rotary_dim=136), BAD),
    (dict(rotary_dim=0), BAD),                                      # positions are given
    (dict(period=0), BAD), (dict(period=-1), BAD), (dict(flags=4), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD), (dict(dtype=3), NOT_OFFERED),
    (dict(dim=12), NOT_OFFERED), (dict(dim=264), NOT_OFFERED),
    (dict(tokens=1 << 30), NOT_OFFERED), (dict(b_heads=(1 << 20) + 1), NOT_OFFERED),
    (dict(b_stride=248), BAD), (dict(c_stride=508), BAD), (dict(b_out_stride=260), BAD),
    (dict(c_out_stride=1 << 31), BAD),
]


@pytest.mark.parametrize("kw,status", NORM_REFUSED)
def test_norm_refuses(lib, kw, status):
    assert _norm(lib, NP(**kw)) == status
    assert _norm_back(lib, NP(**kw)) == status


def test_norm_refuses_pointers(lib):
    off = vp(4096 + 8)
    for k in ("B", "C", "bo", "co"):
        assert _norm(lib, NP(), **{k: None}) == BAD and _norm(lib, NP(), **{k: off}) == BAD, k
    for k in ("dbo", "dco", "B", "C", "dB", "dC"):
        assert _norm_back(lib, NP(), **{k: None}) == BAD, k
        assert _norm_back(lib, NP(), **{k: off}) == BAD, k
    assert _norm(lib, NP(), pos=None) == _norm(lib, NP(), freqs=None) == BAD
    assert _norm(lib, None) == _norm_back(lib, None) == BAD
    for kw in (dict(db_stride=248), dict(dc_stride=500)):
        assert _norm_back(lib, NP(**kw)) == BAD
    n = ctypes.c_size_t(0)
    size = lib.ssd_bc_norm_backward_workspace_size
    assert size(NP(), ctypes.byref(n)) == ssd.SSD_OK and n.value % (2 * 128 * 4) == 0
    assert size(NP(), None) == BAD
    assert _norm_back(lib, NP(), ws=None) == WS
    assert _norm_back(lib, NP(), ws=vp(4096 + 64)) == WS
    assert _norm_back(lib, NP(), wsb=n.value - 1) == WS


def test_norm_without_tokens_is_a_no_op(lib):
    assert _norm(lib, NP(tokens=0), B=None, bo=None) == ssd.SSD_OK
    assert _norm_back(lib, NP(tokens=0), dB=None, dbw=None, dcw=None, ws=None) == ssd.SSD_OK


def test_norm_backward_workspace_is_small(lib):
    n = ctypes.c_size_t(0)
    for tokens in (1, 100, 1 << 20, (1 << 30) - 1):
        assert lib.ssd_bc_norm_backward_workspace_size(NP(tokens=tokens), ctypes.byref(n)) == 0
        assert 0 < n.value <= 1024 * 2 * 128 * 4


# ---- the binding -------------------------------------------------------------------


def _m(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


F32 = torch.float32


def _delta(**kw):
    t = dict(x=_m(2, 9, 4, 64), g=_m(2, 9, 4), beta=_m(2, 9, 4), B=_m(2, 9, 2, 32),
             C=_m(2, 9, 2, 32), initial_state=_m(2, 4, 64, 32, dtype=F32))
    t.update(kw)
    return t


DELTA_BAD = [
    dict(x=_m(2, 9, 256)), dict(x=_m(2, 9, 4, 64, dtype=torch.float16)), dict(B=_m(2, 9, 64)),
    dict(B=_m(2, 8, 2, 32)), dict(C=_m(2, 9, 2, 48)), dict(C=_m(2, 9, 4, 32)),
    dict(g=_m(2, 9, 4, dtype=F32)), dict(g=_m(2, 9, 1)), dict(beta=_m(2, 4, 9)),
    dict(initial_state=_m(2, 4, 64, 32)), dict(initial_state=_m(2, 4, 32, 64, dtype=F32)),
    dict(B=torch.empty(2, 9, 2, 32, dtype=torch.bfloat16)),           # another device
    dict(cu_seqlens=torch.tensor([0, 9], dtype=torch.int32)),         # of a batch of two
]


@pytest.mark.parametrize("kw", DELTA_BAD)
def test_delta_binding_refuses(kw, monkeypatch):
    monkeypatch.setattr(_lib, "_on_gpu", lambda dev: None)
    with pytest.raises(ValueError):
        ssd.delta_forward(**_delta(**kw))
    with pytest.raises(ValueError):
        ssd.delta_backward(dy=_m(2, 9, 4, 64), **_delta(**kw))


@pytest.mark.parametrize("kw", [
    dict(y=_m(2, 9, 4, 32)), dict(y=_m(2, 9, 4, 64, dtype=F32)), dict(y=_m(2, 4, 9, 64).transpose(1, 2)),
    dict(final_state=_m(2, 4, 64, 32)), dict(final_state=_m(1, 4, 64, 32, dtype=F32)),
    dict(final_state=_m(2, 4, 32, 64, dtype=F32).transpose(2, 3)),
])
def test_delta_binding_refuses_outputs(kw, monkeypatch):
    monkeypatch.setattr(_lib, "_on_gpu", lambda dev: None)
    with pytest.raises(ValueError):
        ssd.delta_forward(**_delta(), **kw)


@pytest.mark.parametrize("cu", [[0], [0, 5, 8], [1, 9], [0, 7, 5, 9], [[0, 9]], [0, -1, 9]])
def test_delta_binding_refuses_offsets(cu, monkeypatch):
    monkeypatch.setattr(_lib, "_on_gpu", lambda dev: None)
    t = {k: v[:1] for k, v in _delta(initial_state=_m(1, 4, 64, 32, dtype=F32)).items()}
    with pytest.raises(ValueError):
        ssd.delta_forward(cu_seqlens=torch.tensor(cu, dtype=torch.int32), **t)


def test_delta_binding_refuses_the_rest(monkeypatch):
    with pytest.raises(ValueError):              # not a GPU's tensors
        ssd.delta_forward(**{k: torch.empty(v.shape, dtype=v.dtype) for k, v in _delta().items()})
    monkeypatch.setattr(_lib, "_on_gpu", lambda dev: None)
    for dy in (None, _m(2, 9, 4, 32), _m(2, 9, 4, 64, dtype=F32)):
        with pytest.raises(ValueError):
            ssd.delta_backward(dy=dy, **_delta())
    with pytest.raises(ValueError):
        ssd.delta_backward(dy=_m(2, 9, 4, 64), dfinal_state=_m(2, 4, 64, 32), **_delta())
    one = {k: v[:, 0] for k, v in _delta().items() if k != "initial_state"}
    state = _m(2, 4, 64, 32, dtype=F32)
    for kw in (dict(state=None), dict(state=_m(2, 4, 64, 32)), dict(state=state.transpose(2, 3)),
               dict(state=state[:1]), dict(state=state, y=_m(2, 4, 32)),
               dict(state=state, y=_m(4, 2, 64).transpose(0, 1)), dict(state=state, g=_m(2, 4, 1)),
               dict(state=state, x=_m(2, 9, 4, 64))):
        with pytest.raises(ValueError):
            ssd.delta_step(**dict(one, **kw))


@pytest.mark.parametrize("kw", [
    dict(B=_m(128)), dict(B=_m(5, 2, 128, dtype=torch.float16)), dict(C=_m(6, 4, 128)),
    dict(C=_m(5, 4, 64)), dict(C=_m(5, 4, 128, dtype=F32)), dict(B_weight=_m(128)),
    dict(C_weight=_m(64, dtype=F32)), dict(positions=None), dict(freqs=None),
    dict(freqs=_m(4, 8, dtype=F32)), dict(freqs=_m(32)), dict(positions=_m(5, dtype=F32)),
    dict(positions=_m(4, dtype=torch.int32)), dict(positions=_m(5, 1, dtype=torch.int32)),
    dict(B_out=_m(5, 2, 64)), dict(C_out=_m(5, 4, 128, dtype=F32)),
    dict(C_out=_m(5, 128, 4).transpose(1, 2)), dict(C=torch.empty(5, 4, 128, dtype=torch.bfloat16)),
])
def test_norm_binding_refuses(kw, monkeypatch):
    monkeypatch.setattr(_lib, "_on_gpu", lambda dev: None)
    monkeypatch.setattr(_lib, "_stream_of", lambda dev, stream: (torch.no_grad(), None))
    t = dict(B=_m(5, 2, 128), C=_m(5, 4, 128), B_weight=_m(128, dtype=F32),
             C_weight=_m(128, dtype=F32), positions=_m(5, dtype=torch.int64),
             freqs=_m(32, dtype=F32))
    t.update(kw)
    with pytest.raises(ValueError):
        ssd.bc_norm(**t)
    t = {{"B_out": "dB", "C_out": "dC"}.get(k, k): v for k, v in t.items()}
    with pytest.raises(ValueError):
        ssd.bc_norm_backward(_m(5, 2, 128), _m(5, 4, 128), **t)


def test_norm_binding_needs_gradients(monkeypatch):
    monkeypatch.setattr(_lib, "_on_gpu", lambda dev: None)
    B, C = _m(5, 2, 128), _m(5, 4, 128)
    for d in ((None, C), (B, None), (C, C), (B, B)):
        with pytest.raises(ValueError):
            ssd.bc_norm_backward(*d, B, C)
    with pytest.raises(ValueError):              # not a GPU's tensors
        monkeypatch.undo()
        ssd.bc_norm(torch.empty(5, 2, 128), torch.empty(5, 4, 128))
