"""ctypes binding of ``libssd.so`` (declared in ``include/ssd.h``).

Argument marshalling only: torch provides device memory and the current HIP
stream; every step of the SSD forward pass runs in the library's kernels.
There is no CPU fallback -- if the library is missing, import succeeds but
every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssd.so")

SSD_OK, SSD_ERR_INVALID_ARG, SSD_ERR_UNSUPPORTED, SSD_ERR_WORKSPACE, SSD_ERR_HIP = range(5)
SSD_DTYPE_F32, SSD_DTYPE_BF16 = 0, 1
SSD_FLAG_GENERIC_KERNELS = 1
SSD_FLAG_UNFUSED = 2
SSD_FLAG_PER_SEQUENCE = 4
SSD_NORM_CENTER, SSD_NORM_BEFORE_GATE = 1, 2
CHECKPOINT_BLOCK = 32   # channels that share a scale in an 8-bit checkpoint


class SSDError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__("%s: %s (%s)" % (where, _status_string(status), detail))


class Problem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32),
                ("nheads", ctypes.c_int32), ("headdim", ctypes.c_int32),
                ("dstate", ctypes.c_int32), ("ngroups", ctypes.c_int32),
                ("chunk_size", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]

    def __repr__(self):
        return "Problem(%s)" % ", ".join("%s=%s" % (f, getattr(self, f)) for f, _ in self._fields_)


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [("chunk_cumsum", ctypes.c_size_t), ("chunk_states", ctypes.c_size_t),
                ("chunk_table", ctypes.c_size_t), ("chunk_records", ctypes.c_int64),
                ("max_chunks", ctypes.c_int64), ("chain_sync", ctypes.c_size_t),
                ("chain_sync_words", ctypes.c_int64), ("chain_chunks_per_unit", ctypes.c_int64),
                ("chain_ranges", ctypes.c_int64)]


class ScanProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("dstate", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class ConvProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("x_dim", ctypes.c_int32),
                ("bc_dim", ctypes.c_int32), ("width", ctypes.c_int32),
                ("in_stride", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class NormProblem(ctypes.Structure):
    _fields_ = [("x_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("dx_stride", ctypes.c_int64),
                ("dz_stride", ctypes.c_int64),
                ("tokens", ctypes.c_int32), ("channels", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("eps", ctypes.c_float)]


class CheckpointProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("stride", ctypes.c_int64),
                ("channels", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class CheckpointArg(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("exponents", ctypes.c_void_p)]


MAX_STAGES = 12


class StageTimes(ctypes.Structure):
    _fields_ = [("num_stages", ctypes.c_int32), ("iterations", ctypes.c_int32),
                ("names", (ctypes.c_char * 24) * MAX_STAGES),
                ("ms", ctypes.c_float * MAX_STAGES), ("total_ms", ctypes.c_float)]

    def as_dict(self):
        """{kernel name: mean ms per launch}, plus '_total_ms' (all iterations)."""
        out = {self.names[k].value.decode(): self.ms[k] / max(self.iterations, 1)
               for k in range(self.num_stages)}
        out["_total_ms"] = self.total_ms
        return out


EXPORTED = ("ssd_validate", "ssd_validate_cu_seqlens", "ssd_workspace_size",
            "ssd_forward", "ssd_forward_noalloc", "ssd_forward_dt_softplus",
            "ssd_forward_timed", "ssd_step",
            "ssd_selective_scan", "ssd_conv1d_silu",
            "ssd_backward_workspace_size", "ssd_backward", "ssd_backward_timed",
            "ssd_conv1d_silu_checkpoint", "ssd_conv1d_silu_backward_workspace_size",
            "ssd_conv1d_silu_backward", "ssd_group_norm_silu",
            "ssd_group_norm_silu_backward_workspace_size", "ssd_group_norm_silu_backward",
            "ssd_checkpoint_save", "ssd_checkpoint_load",
            "ssd_get_workspace_layout",
            "ssd_status_string", "ssd_last_error_detail")

_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Load libssd.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                "libssd.so is not built (%s); run `python -m mamba_ssd_sequence_fwd_amd.build`"
                % path)
        lib = ctypes.CDLL(path)
        P = ctypes.POINTER(Problem)
        vp = ctypes.c_void_p
        lib.ssd_validate.argtypes = [P]
        lib.ssd_validate_cu_seqlens.argtypes = [P, vp]
        lib.ssd_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        lib.ssd_get_workspace_layout.argtypes = [P, ctypes.POINTER(WorkspaceLayout)]
        lib.ssd_forward.argtypes = [P] + [vp] * 11 + [ctypes.c_size_t, vp]
        lib.ssd_forward_noalloc.argtypes = [P] + [vp] * 11
        lib.ssd_forward_timed.argtypes = ([P] + [vp] * 11 + [ctypes.c_size_t, vp, ctypes.c_int32,
                                          ctypes.POINTER(StageTimes)])
        lib.ssd_step.argtypes = [P] + [vp] * 9
        lib.ssd_forward_dt_softplus.argtypes = [P] + [vp] * 12 + [ctypes.c_size_t, vp]
        lib.ssd_selective_scan.argtypes = [ctypes.POINTER(ScanProblem)] + [vp] * 10
        lib.ssd_conv1d_silu.argtypes = [ctypes.POINTER(ConvProblem)] + [vp] * 10
        CV, NM = ctypes.POINTER(ConvProblem), ctypes.POINTER(NormProblem)
        KP, KA = ctypes.POINTER(CheckpointProblem), ctypes.POINTER(CheckpointArg)
        szp = ctypes.POINTER(ctypes.c_size_t)
        lib.ssd_conv1d_silu_checkpoint.argtypes = [CV, vp, KA] + [vp] * 9
        lib.ssd_conv1d_silu_backward_workspace_size.argtypes = [CV, szp]
        lib.ssd_conv1d_silu_backward.argtypes = ([CV, vp, KA] + [vp] * 9 + [ctypes.c_int32]
                                                 + [vp] * 4 + [ctypes.c_size_t, vp])
        lib.ssd_group_norm_silu.argtypes = [NM] + [vp] * 5 + [KA, KA, vp]
        lib.ssd_group_norm_silu_backward_workspace_size.argtypes = [NM, szp]
        lib.ssd_group_norm_silu_backward.argtypes = ([NM] + [vp] * 3 + [KA, KA] + [vp] * 7
                                                     + [ctypes.c_size_t, vp])
        lib.ssd_checkpoint_save.argtypes = [KP, vp, KA, vp]
        lib.ssd_checkpoint_load.argtypes = [KP, KA, vp, vp]
        lib.ssd_backward_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        lib.ssd_backward.argtypes = [P] + [vp] * 18 + [ctypes.c_size_t, vp]
        lib.ssd_backward_timed.argtypes = ([P] + [vp] * 18 + [ctypes.c_size_t, vp,
                                           ctypes.c_int32, ctypes.POINTER(StageTimes)])
        for f in ("ssd_validate", "ssd_validate_cu_seqlens", "ssd_workspace_size",
                  "ssd_get_workspace_layout", "ssd_forward", "ssd_forward_noalloc",
                  "ssd_forward_timed", "ssd_step",
                  "ssd_selective_scan", "ssd_forward_dt_softplus"):
            getattr(lib, f).restype = ctypes.c_int
        lib.ssd_status_string.argtypes = [ctypes.c_int]
        lib.ssd_status_string.restype = ctypes.c_char_p
        lib.ssd_last_error_detail.argtypes = []
        lib.ssd_last_error_detail.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _status_string(st: int) -> str:
    try:
        return load().ssd_status_string(st).decode()
    except Exception:  # pragma: no cover - only while reporting another error
        return "status %d" % st


def _check(st: int, where: str):
    if st != SSD_OK:
        raise SSDError(st, where, load().ssd_last_error_detail().decode())


def make_problem(batch, seqlen, nheads, headdim, dstate, ngroups, chunk_size,
                 num_seqs=0, dtype=SSD_DTYPE_BF16, flags=0) -> Problem:
    return Problem(batch, seqlen, nheads, headdim, dstate, ngroups, chunk_size,
                   num_seqs, dtype, flags)


def validate(prob: Problem):
    _check(load().ssd_validate(ctypes.byref(prob)), "ssd_validate")


def validate_cu_seqlens(prob: Problem, cu_host):
    cu = torch.as_tensor(cu_host, dtype=torch.int32).contiguous().cpu()
    _check(load().ssd_validate_cu_seqlens(ctypes.byref(prob), ctypes.c_void_p(cu.data_ptr())),
           "ssd_validate_cu_seqlens")


def workspace_size(prob: Problem) -> int:
    n = ctypes.c_size_t(0)
    _check(load().ssd_workspace_size(ctypes.byref(prob), ctypes.byref(n)), "ssd_workspace_size")
    return int(n.value)


def workspace_layout(prob: Problem) -> WorkspaceLayout:
    lay = WorkspaceLayout()
    _check(load().ssd_get_workspace_layout(ctypes.byref(prob), ctypes.byref(lay)),
           "ssd_get_workspace_layout")
    return lay


_DTYPES = {torch.bfloat16: SSD_DTYPE_BF16, torch.float32: SSD_DTYPE_F32}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _same_device(dev, **tensors):
    """Every tensor a kernel reads or writes must live on ``dev`` (the device
    of the first input): a host pointer handed to a kernel would fault the GPU
    instead of raising. Checked before anything is launched."""
    for name, t in tensors.items():
        if t is not None:
            if isinstance(t, Checkpoint):
                _refuse_checkpoint(name)
            if t.device != dev:
                raise ValueError("%s is on %s, but the other inputs are on %s"
                                 % (name, t.device, dev))


def _refuse_checkpoint(name):
    """A Checkpoint (which has a tensor's shape, dtype and device) where a tensor belongs."""
    raise ValueError("%s is a Checkpoint, but must be a tensor (load() gives its values)" % name)


def _on_gpu(dev):
    if dev.type != "cuda":
        raise ValueError("tensors must be on the GPU (got %s)" % dev)


class Plan:
    """A prepared ssd_forward call: validated problem, outputs and workspace
    allocated once; :meth:`run` only enqueues the kernels.

    Shapes: x (batch, L, H, P); dt (batch, L, H); A (H,) fp32; B, C
    (batch, L, G, N); D (H,) fp32 or None; initial_state (batch | num_seqs,
    H, P, N) fp32 or None; cu_seqlens (num_seqs + 1,) int32 (CPU or GPU) or
    None. x, dt, B, C share the dtype (bfloat16 or float32).

    With ``dt_softplus=True`` dt holds the step's pre-activation and the
    kernels use softplus(dt + dt_bias[h]) (ssd_forward_dt_softplus); dt_bias
    is (H,) fp32 or None.
    """

    def __init__(self, x, dt, A, B, C, D=None, initial_state=None, chunk_size=256,
                 cu_seqlens=None, *, want_final_state=True, generic=False,
                 unfused=False, per_sequence=False, check_cu_seqlens=True,
                 dt_softplus=False, dt_bias=None):
        if x.dim() != 4:
            raise ValueError("x must be (batch, seqlen, nheads, headdim)")
        batch, L, H, P = x.shape
        G, N = B.shape[2], B.shape[3]
        dev = x.device
        _same_device(dev, dt=dt, A=A, B=B, C=C, D=D, initial_state=initial_state,
                     dt_bias=dt_bias)
        _on_gpu(dev)
        if x.dtype not in _DTYPES:
            raise ValueError("x must be bfloat16 or float32")
        for name, t, shape in (("dt", dt, (batch, L, H)), ("B", B, (batch, L, G, N)),
                               ("C", C, (batch, L, G, N))):
            if tuple(t.shape) != shape or t.dtype != x.dtype or t.device != dev:
                raise ValueError("%s must be %s %s on %s" % (name, shape, x.dtype, dev))
        if tuple(A.shape) != (H,) or A.dtype != torch.float32:
            raise ValueError("A must be (H,) float32")
        if D is not None and (tuple(D.shape) != (H,) or D.dtype != torch.float32):
            raise ValueError("D must be (H,) float32")
        num_seqs = 0
        cu_dev = None
        if cu_seqlens is not None:
            if batch != 1:
                raise ValueError("cu_seqlens needs batch == 1")
            num_seqs = int(cu_seqlens.numel()) - 1
        nstate = num_seqs if num_seqs else batch
        if initial_state is not None and (
                tuple(initial_state.shape) != (nstate, H, P, N)
                or initial_state.dtype != torch.float32):
            raise ValueError("initial_state must be (%d, %d, %d, %d) float32" % (nstate, H, P, N))
        self.prob = make_problem(batch, L, H, P, N, G, chunk_size, num_seqs,
                                 _DTYPES[x.dtype],
                                 (SSD_FLAG_GENERIC_KERNELS if generic else 0)
                                 | (SSD_FLAG_UNFUSED if unfused else 0)
                                 | (SSD_FLAG_PER_SEQUENCE if per_sequence else 0))
        validate(self.prob)
        if cu_seqlens is not None:
            if check_cu_seqlens or cu_seqlens.device.type == "cpu":
                validate_cu_seqlens(self.prob, cu_seqlens.detach().cpu())
            cu_dev = cu_seqlens.to(device=dev, dtype=torch.int32).contiguous()
        if dt_bias is not None:
            if not dt_softplus:
                raise ValueError("dt_bias needs dt_softplus=True")
            if tuple(dt_bias.shape) != (H,) or dt_bias.dtype != torch.float32 or dt_bias.device != dev:
                raise ValueError("dt_bias must be (H,) float32 on %s" % dev)
            dt_bias = dt_bias.contiguous()
        self.dt_softplus = bool(dt_softplus)
        self.dt_bias = dt_bias
        self.inputs = [t.contiguous() if t is not None else None
                       for t in (x, dt, A, B, C, D, initial_state)]
        self.cu = cu_dev
        self.y = torch.empty_like(x)
        self.final_state = (torch.empty((nstate, H, P, N), device=dev, dtype=torch.float32)
                            if want_final_state else None)
        self.ws_bytes = workspace_size(self.prob)
        self.workspace = torch.empty(max(self.ws_bytes, 256), device=dev, dtype=torch.uint8)
        self.tokens = batch * L

    def run(self, stream=None):
        """Enqueue one forward pass on ``stream`` (default: torch's current)."""
        if stream is None:
            stream = torch.cuda.current_stream(self.y.device)
        x, dt, A, B, C, D, h0 = self.inputs
        if self.dt_softplus:
            _check(load().ssd_forward_dt_softplus(
                ctypes.byref(self.prob), _ptr(x), _ptr(dt), _ptr(self.dt_bias), _ptr(A),
                _ptr(B), _ptr(C), _ptr(D), _ptr(h0), _ptr(self.cu), _ptr(self.y),
                _ptr(self.final_state), _ptr(self.workspace),
                ctypes.c_size_t(self.workspace.numel()), ctypes.c_void_p(stream.cuda_stream)),
                "ssd_forward_dt_softplus")
            return self.y, self.final_state
        _check(load().ssd_forward(
            ctypes.byref(self.prob), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
            _ptr(D), _ptr(h0), _ptr(self.cu), _ptr(self.y), _ptr(self.final_state),
            _ptr(self.workspace), ctypes.c_size_t(self.workspace.numel()),
            ctypes.c_void_p(stream.cuda_stream)), "ssd_forward")
        return self.y, self.final_state

    def run_timed(self, iterations: int, stream=None) -> StageTimes:
        """``iterations`` passes with a HIP event after every kernel; waits for
        them and returns the per-kernel times (see ssd_forward_timed)."""
        if self.dt_softplus:
            raise ValueError("run_timed times ssd_forward; it has no raw-step variant")
        if stream is None:
            stream = torch.cuda.current_stream(self.y.device)
        x, dt, A, B, C, D, h0 = self.inputs
        times = StageTimes()
        _check(load().ssd_forward_timed(
            ctypes.byref(self.prob), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
            _ptr(D), _ptr(h0), _ptr(self.cu), _ptr(self.y), _ptr(self.final_state),
            _ptr(self.workspace), ctypes.c_size_t(self.workspace.numel()),
            ctypes.c_void_p(stream.cuda_stream), int(iterations), ctypes.byref(times)),
            "ssd_forward_timed")
        return times

    def layout(self) -> WorkspaceLayout:
        return workspace_layout(self.prob)

    def chain_error(self) -> int:
        """Error word of the chained kernel after the passes run so far
        (synchronises): nonzero if a workgroup gave up waiting for its
        predecessor's state. 0 when the problem does not use that kernel."""
        lay = self.layout()
        if lay.chain_sync_words == 0:
            return 0
        torch.cuda.synchronize(self.workspace.device)
        w = self.workspace[lay.chain_sync:lay.chain_sync + 8].view(torch.int32)
        return int(w[1].item())

    def check(self):
        """Wait for the passes run so far and raise SSDError if the chained
        kernel's error word is set (see :meth:`chain_error`)."""
        err = self.chain_error()
        if err:
            raise SSDError(SSD_ERR_HIP, "ssd_forward",
                           "a chained workgroup timed out waiting for its predecessor's "
                           "state (error word %d); the outputs are invalid" % err)


def forward(x, dt, A, B, C, D=None, initial_state=None, chunk_size=256, cu_seqlens=None,
            *, check=False, **kw):
    """SSD forward pass: returns (y, final_state).

    With ``check=True`` the call waits for the pass and raises SSDError if a
    chained workgroup gave up waiting for its predecessor's state (the error
    word of the workspace; the outputs are then wrong)."""
    plan = Plan(x, dt, A, B, C, D, initial_state, chunk_size, cu_seqlens, **kw)
    y, hT = plan.run()
    if check:
        plan.check()
    return y, hT


def forward_noalloc(x, dt, A, B, C, D, initial_state, y, final_state, chunk_size=256,
                    cu_seqlens=None, *, stream=None):
    """ssd_forward_noalloc: the forward pass into caller-provided ``y`` and
    ``final_state`` (or None) with the library's fixed device scratch area as
    the workspace; nothing is allocated. Tensors as for :class:`Plan`, all on
    one GPU; ``cu_seqlens`` int32 on that GPU (no host copy, no check of its
    values here). Calls that may overlap on one GPU race on the scratch area.
    """
    if x.dim() != 4:
        raise ValueError("x must be (batch, seqlen, nheads, headdim)")
    batch, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    _same_device(dev, dt=dt, A=A, B=B, C=C, D=D, initial_state=initial_state, y=y,
                 final_state=final_state, cu_seqlens=cu_seqlens)
    _on_gpu(dev)
    if x.dtype not in _DTYPES:
        raise ValueError("x must be bfloat16 or float32")
    num_seqs = 0 if cu_seqlens is None else int(cu_seqlens.numel()) - 1
    if cu_seqlens is not None and (cu_seqlens.dtype != torch.int32 or batch != 1):
        raise ValueError("cu_seqlens must be int32 with batch == 1")
    nstate = num_seqs if num_seqs else batch
    for name, t, shape, dtype in (
            ("dt", dt, (batch, L, H), x.dtype), ("B", B, (batch, L, G, N), x.dtype),
            ("C", C, (batch, L, G, N), x.dtype), ("A", A, (H,), torch.float32),
            ("D", D, (H,), torch.float32), ("y", y, (batch, L, H, P), x.dtype),
            ("initial_state", initial_state, (nstate, H, P, N), torch.float32),
            ("final_state", final_state, (nstate, H, P, N), torch.float32)):
        if t is None and name in ("dt", "B", "C", "A", "y"):
            raise ValueError("%s is required" % name)
        if t is not None and (tuple(t.shape) != shape or t.dtype != dtype
                              or not t.is_contiguous()):
            raise ValueError("%s must be a contiguous %s %s tensor" % (name, shape, dtype))
    for name, t in (("x", x), ("cu_seqlens", cu_seqlens)):
        if t is not None and not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    prob = make_problem(batch, L, H, P, N, G, chunk_size, num_seqs, _DTYPES[x.dtype], 0)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    _check(load().ssd_forward_noalloc(
        ctypes.byref(prob), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
        _ptr(initial_state), _ptr(cu_seqlens), _ptr(y), _ptr(final_state),
        ctypes.c_void_p(stream.cuda_stream)), "ssd_forward_noalloc")
    return y, final_state


def step(x, dt, A, B, C, D=None, state=None, *, y=None, stream=None):
    """One decode step (ssd_step): every sequence advances by one token and
    ``state`` is updated IN PLACE; returns y.

    Shapes: x (batch, H, P); dt (batch, H); A (H,) fp32; B, C (batch, G, N);
    D (H,) fp32 or None; state (batch, H, P, N) fp32, contiguous; y (optional
    output) like x. x, dt, B, C share the dtype (bfloat16 or float32).
    """
    if x.dim() != 3:
        raise ValueError("x must be (batch, nheads, headdim)")
    batch, H, P = x.shape
    if B.dim() != 3:
        raise ValueError("B must be (batch, ngroups, dstate)")
    G, N = B.shape[1], B.shape[2]
    dev = x.device
    _same_device(dev, dt=dt, A=A, B=B, C=C, D=D, state=state, y=y)
    _on_gpu(dev)
    if x.dtype not in _DTYPES:
        raise ValueError("x must be bfloat16 or float32")
    for name, t, shape in (("dt", dt, (batch, H)), ("B", B, (batch, G, N)),
                           ("C", C, (batch, G, N))):
        if tuple(t.shape) != shape or t.dtype != x.dtype or t.device != dev:
            raise ValueError("%s must be %s %s on %s" % (name, shape, x.dtype, dev))
    if tuple(A.shape) != (H,) or A.dtype != torch.float32:
        raise ValueError("A must be (H,) float32")
    if D is not None and (tuple(D.shape) != (H,) or D.dtype != torch.float32):
        raise ValueError("D must be (H,) float32")
    if (state is None or tuple(state.shape) != (batch, H, P, N)
            or state.dtype != torch.float32 or not state.is_contiguous()
            or state.device != dev):
        raise ValueError("state must be a contiguous (%d, %d, %d, %d) float32 tensor on %s"
                         % (batch, H, P, N, dev))
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif tuple(y.shape) != (batch, H, P) or y.dtype != x.dtype or not y.is_contiguous():
        raise ValueError("y must be a contiguous (%d, %d, %d) %s tensor" % (batch, H, P, x.dtype))
    prob = make_problem(batch, 1, H, P, N, G, 0, 0, _DTYPES[x.dtype], 0)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    # copies of non-contiguous inputs are made on the stream the kernel runs
    # on, so they are complete before it reads them and their memory is not
    # reused before it has run
    with torch.cuda.stream(stream):
        x, dt, A, B, C = (t.contiguous() for t in (x, dt, A, B, C))
        D = D.contiguous() if D is not None else None
    _check(load().ssd_step(ctypes.byref(prob), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                           _ptr(D), _ptr(state), _ptr(y), ctypes.c_void_p(stream.cuda_stream)),
           "ssd_step")
    return y


def selective_scan(x, delta, A, B, C, D=None, initial_state=None, *, want_final_state=True,
                   y=None, final_state=None, stream=None):
    """The Mamba-1 selective scan (ssd_selective_scan): returns (y, final_state).

    Shapes: x, delta (batch, L, dim); A (dim, N) fp32; B, C (batch, L, N);
    D (dim,) fp32 or None; initial_state (batch, dim, N) fp32 or None. x,
    delta, B, C share the dtype (bfloat16 or float32); dim must be a multiple
    of 64 and N one of 16, 32, 64, 128, 256.
    """
    if x.dim() != 3:
        raise ValueError("x must be (batch, seqlen, dim)")
    batch, L, Dm = x.shape
    if A.dim() != 2 or A.shape[0] != Dm or A.dtype != torch.float32:
        raise ValueError("A must be (dim, dstate) float32")
    N = A.shape[1]
    dev = x.device
    _same_device(dev, delta=delta, A=A, B=B, C=C, D=D, initial_state=initial_state, y=y,
                 final_state=final_state)
    _on_gpu(dev)
    if x.dtype not in _DTYPES:
        raise ValueError("x must be bfloat16 or float32")
    for name, t, shape in (("delta", delta, (batch, L, Dm)), ("B", B, (batch, L, N)),
                           ("C", C, (batch, L, N))):
        if tuple(t.shape) != shape or t.dtype != x.dtype or t.device != dev:
            raise ValueError("%s must be %s %s on %s" % (name, shape, x.dtype, dev))
    if D is not None and (tuple(D.shape) != (Dm,) or D.dtype != torch.float32):
        raise ValueError("D must be (dim,) float32")
    if initial_state is not None and (tuple(initial_state.shape) != (batch, Dm, N)
                                      or initial_state.dtype != torch.float32):
        raise ValueError("initial_state must be (%d, %d, %d) float32" % (batch, Dm, N))
    prob = ScanProblem(batch, L, Dm, N, _DTYPES[x.dtype], 0)
    if y is not None and (tuple(y.shape) != (batch, L, Dm) or y.dtype != x.dtype
                          or not y.is_contiguous()):
        raise ValueError("y must be a contiguous (%d, %d, %d) %s tensor" % (batch, L, Dm, x.dtype))
    if final_state is not None and (tuple(final_state.shape) != (batch, Dm, N)
                                    or final_state.dtype != torch.float32
                                    or not final_state.is_contiguous()):
        raise ValueError("final_state must be a contiguous (%d, %d, %d) float32 tensor"
                         % (batch, Dm, N))
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    # copies and outputs are made on the stream the kernel runs on (see step())
    with torch.cuda.stream(stream):
        x, delta, A, B, C = (t.contiguous() for t in (x, delta, A, B, C))
        D = D.contiguous() if D is not None else None
        h0 = initial_state.contiguous() if initial_state is not None else None
        if y is None:
            y = torch.empty_like(x)
        if final_state is None and want_final_state:
            final_state = torch.empty((batch, Dm, N), device=dev, dtype=torch.float32)
    _check(load().ssd_selective_scan(ctypes.byref(prob), _ptr(x), _ptr(delta), _ptr(A), _ptr(B),
                                     _ptr(C), _ptr(D), _ptr(h0), _ptr(y), _ptr(final_state),
                                     ctypes.c_void_p(stream.cuda_stream)),
           "ssd_selective_scan")
    return y, final_state


class Checkpoint:
    """An activation kept in 8 bits between the forward and the backward pass.

    ``q`` (..., channels) int8 and ``exponents`` (..., ceil(channels / 32))
    uint8, both contiguous, channels a multiple of 8: an element's value is
    ``q * 2**(exponent of its block of 32 channels - 127)``, within half a step
    of what was saved (a block that held an infinity or NaN reads as NaN).
    ``dtype`` is the dtype of the tensor it stands for (bfloat16 or float32).
    Written by :func:`checkpoint_save`, :func:`conv1d_silu` and
    :func:`group_norm_silu`; read by :meth:`load`, :func:`conv1d_silu` and the
    backward functions.
    """
    __slots__ = ("q", "exponents", "dtype")

    def __init__(self, q, exponents, dtype):
        if dtype not in _DTYPES:
            raise ValueError("a checkpoint stands for a bfloat16 or float32 tensor")
        if q.dim() < 1 or q.dtype != torch.int8 or not q.is_contiguous():
            raise ValueError("q must be a contiguous int8 tensor")
        if q.shape[-1] < 8 or q.shape[-1] % 8 != 0:
            raise ValueError("channels (%d) must be a multiple of 8" % q.shape[-1])
        shape = q.shape[:-1] + (-(-q.shape[-1] // CHECKPOINT_BLOCK),)
        if (exponents.shape != shape or exponents.dtype != torch.uint8
                or not exponents.is_contiguous() or exponents.device != q.device):
            raise ValueError("exponents must be a contiguous %s uint8 tensor on %s"
                             % (tuple(shape), q.device))
        self.q, self.exponents, self.dtype = q, exponents, dtype

    @property
    def shape(self):
        return self.q.shape

    @property
    def device(self):
        return self.q.device

    @property
    def nbytes(self):
        return self.q.numel() + self.exponents.numel()

    def arg(self):
        return CheckpointArg(self.q.data_ptr(), self.exponents.data_ptr())

    def load(self, *, out=None, stream=None):
        """The values, in ``dtype`` (exact; see ssd_checkpoint_load), in a new
        tensor or in ``out`` (rows may be a slice of wider rows)."""
        dev, ch = self.q.device, self.q.shape[-1]
        if out is not None:
            _same_device(dev, out=out)
        _on_gpu(dev)
        context, handle = _stream_of(dev, stream)
        with context:
            if out is None:
                out = self.q.new_empty(self.q.shape, dtype=self.dtype)
            elif out.shape != self.q.shape or out.dtype != self.dtype:
                raise ValueError("out must be %s %s" % (tuple(self.q.shape), self.dtype))
            stride = _stride_of_out(out, "out")
            prob = CheckpointProblem(out.numel() // ch, stride, ch, _DTYPES[self.dtype], 0)
            _check(load().ssd_checkpoint_load(prob, self.arg(), out.data_ptr(), handle),
                   "ssd_checkpoint_load")
        return out


_NO_CONTEXT = contextlib.nullcontext()
# The handle of the current stream of a device, without the Stream object that
# torch.cuda.current_stream makes around it (2 us of a call of 9 to 19).
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream_of(dev, stream):
    """(context, handle) of the stream to launch on: torch's current one on
    ``dev``, or the caller's, which must be one of that device. Copies, outputs
    and workspaces made in the context belong to that stream, and ``dev`` is
    the current device in it; none is needed where both are so already."""
    if stream is None:
        if torch.cuda.current_device() == dev.index:
            return _NO_CONTEXT, _current_handle(dev.index)
        stream = torch.cuda.current_stream(dev)
    elif stream.device != dev:
        raise ValueError("the stream is on %s, but the tensors are on %s" % (stream.device, dev))
    return torch.cuda.stream(stream), stream.cuda_stream


# The C structures hold sizes in 32 bits, into which ctypes would wrap larger
# ones; the library itself takes fewer tokens than this.
_MOST_TOKENS = 1 << 30


def _dense(t):
    """``t``, or a copy where it is not contiguous or not 16-byte aligned."""
    if t is None or (t.is_contiguous() and not t.data_ptr() & 15):
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _addr(t):
    return None if t is None else t.data_ptr()


def _row_stride(t):
    """Elements between the token rows of ``t`` (the last axis one row, its
    elements contiguous, all leading axes one evenly spaced sequence of rows,
    16-byte aligned), or None if the rows are not laid out like that."""
    if t.data_ptr() & 15:
        return None
    if t.is_contiguous():
        return t.shape[-1]
    ch = t.shape[-1]
    if t.stride(-1) != 1 and ch > 1:
        return None
    step, rows = None, 1
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if step is None:
            step = stride
        elif stride != step * rows:
            return None
        rows *= size
    step = ch if step is None else step
    return step if step >= ch and step * t.element_size() % 16 == 0 else None


def _stride_of_out(t, name):
    """The row stride of an output, whose rows must be addressable as they are."""
    stride = _row_stride(t)
    if stride is None:
        raise ValueError("the token rows of %s must be evenly spaced, with contiguous channels, "
                         "16-byte aligned" % name)
    return stride


def _rows_in(t):
    """``t`` (or a contiguous copy, where its rows cannot be addressed as they
    are) and its row stride; called on the stream the kernel runs on."""
    stride = _row_stride(t)
    if stride is not None:
        return t, stride
    t = t.clone(memory_format=torch.contiguous_format)
    return t, t.shape[-1]


def _checkpoint_out(given, shape, dtype, dev):
    """The Checkpoint a call fills: a new one for True, or the caller's."""
    if given is True:
        if shape[-1] % 8:
            raise ValueError("channels (%d) must be a multiple of 8" % shape[-1])
        new = object.__new__(Checkpoint)        # (nothing of it needs checking)
        new.q = torch.empty(shape, device=dev, dtype=torch.int8)
        new.exponents = torch.empty(shape[:-1] + (-(-shape[-1] // CHECKPOINT_BLOCK),), device=dev,
                                    dtype=torch.uint8)
        new.dtype = dtype
        return new
    if not isinstance(given, Checkpoint):
        raise ValueError("checkpoint must be True, False or a Checkpoint to fill")
    if tuple(given.shape) != tuple(shape) or given.dtype != dtype or given.device != dev:
        raise ValueError("the checkpoint to fill must be %s for %s on %s"
                         % (tuple(shape), dtype, dev))
    return given


def checkpoint_save(t, *, checkpoint=True, stream=None):
    """Keep tensor ``t`` (..., channels) in 8 bits (ssd_checkpoint_save): returns
    a new :class:`Checkpoint`, or fills the one given. ``t`` is bfloat16 or
    float32, channels a multiple of 8; its rows may be a slice of wider rows."""
    if isinstance(t, Checkpoint):
        _refuse_checkpoint("tensor")
    _on_gpu(t.device)
    if t.dim() < 1 or t.dtype not in _DTYPES:
        raise ValueError("the tensor must be bfloat16 or float32 with a channel axis")
    if t.shape[-1] < 8 or t.shape[-1] % 8 != 0:
        raise ValueError("channels (%d) must be a multiple of 8" % t.shape[-1])
    dev = t.device
    context, handle = _stream_of(dev, stream)
    with context:
        ck = _checkpoint_out(checkpoint, tuple(t.shape), t.dtype, dev)
        t, stride = _rows_in(t)
        prob = CheckpointProblem(t.numel() // t.shape[-1], stride, t.shape[-1],
                                 _DTYPES[t.dtype], 0)
        _check(load().ssd_checkpoint_save(prob, t.data_ptr(), ck.arg(), handle),
               "ssd_checkpoint_save")
    return ck


def _check_offsets(cu, tokens: int):
    """Host check of packed offsets: 0 = cu[0] <= ... <= cu[-1] = tokens."""
    c = cu.detach().to("cpu", torch.int64)
    if c.dim() != 1 or c.numel() < 2 or int(c[0]) != 0 or int(c[-1]) != tokens or \
            bool((c[1:] < c[:-1]).any()):
        raise ValueError("cu_seqlens must rise from 0 to the token count %d" % tokens)


def conv1d_silu(xbc, weight, bias, x_dim, bc_dim, history=None, cu_seqlens=None, *,
                want_history=True, x=None, B=None, C=None, history_out=None,
                checkpoint=False, check_cu_seqlens=True, stream=None):
    """The convolution front (ssd_conv1d_silu): causal depthwise conv1d over
    the packed channels [x | B | C], then SiLU. Returns (x, B, C,
    history_out).

    With ``checkpoint=True`` (or a :class:`Checkpoint` of xbc's shape to fill)
    the call also keeps xbc in 8 bits on the way and returns that Checkpoint
    as a fifth value. xbc may itself be a Checkpoint: x, B and C are then
    recomputed from its values in its dtype, as the backward pass needs them,
    and history_out is None.

    xbc is (batch, L, ch) (dense) or (tokens, ch) with ``cu_seqlens``, ch =
    x_dim + 2 * bc_dim, channels contiguous; its rows may be a slice of wider
    rows (the row stride is passed through). weight (ch, K) and bias (ch,) are
    float32; history (sequences, K - 1, ch) in xbc's dtype or None. Outputs
    have xbc's leading shape with x_dim, bc_dim, bc_dim channels.
    """
    kept = xbc if isinstance(xbc, Checkpoint) else None
    if kept is not None:
        if checkpoint is not False:
            raise ValueError("xbc is a checkpoint already")
        if history_out is not None:
            raise ValueError("a checkpoint does not hold the exact history_out")
        want_history = False
        dtype, xbc = kept.dtype, kept.q
    else:
        dtype = xbc.dtype
        if isinstance(checkpoint, Checkpoint):
            _same_device(xbc.device, checkpoint=checkpoint.q)
    _same_device(xbc.device, weight=weight, bias=bias, history=history, x=x, B=B, C=C,
                 history_out=history_out)
    _on_gpu(xbc.device)
    if dtype not in _DTYPES:
        raise ValueError("xbc must be bfloat16 or float32")
    ch = x_dim + 2 * bc_dim
    if xbc.shape[-1] != ch or xbc.stride(-1) != 1:
        raise ValueError("xbc must end in %d contiguous channels" % ch)
    dev = xbc.device
    if cu_seqlens is not None:
        if xbc.dim() != 2:
            raise ValueError("packed xbc must be (tokens, channels)")
        batch, L = 1, int(xbc.shape[0])
        num_seqs = int(cu_seqlens.numel()) - 1
        if check_cu_seqlens or cu_seqlens.device.type == "cpu":
            _check_offsets(cu_seqlens, L)
        nseq, lead = num_seqs, (L,)
        in_stride = xbc.stride(0) if L > 1 else ch
    else:
        if xbc.dim() != 3:
            raise ValueError("dense xbc must be (batch, seqlen, channels)")
        batch, L = int(xbc.shape[0]), int(xbc.shape[1])
        num_seqs, nseq, lead = 0, batch, (batch, L)
        # token row t = b * L + l sits at b * stride(0) + l * stride(1)
        if L > 1:
            if batch > 1 and xbc.stride(0) != L * xbc.stride(1):
                raise ValueError("the token rows of xbc must be evenly spaced")
            in_stride = xbc.stride(1)
        else:
            in_stride = xbc.stride(0) if batch > 1 else ch
    if batch * L >= 1 << 31 or nseq >= 1 << 31 or in_stride >= 1 << 31:
        raise ValueError("%d tokens in %d sequences, %d elements apart, are more than one call "
                         "takes" % (batch * L, nseq, in_stride))
    K = int(weight.shape[1]) if weight.dim() == 2 else 0
    if tuple(weight.shape) != (ch, K) or weight.dtype != torch.float32:
        raise ValueError("weight must be (%d, K) float32" % ch)
    if bias is not None and (tuple(bias.shape) != (ch,) or bias.dtype != torch.float32):
        raise ValueError("bias must be (%d,) float32" % ch)
    hshape = (nseq, K - 1, ch)
    if history is not None and (tuple(history.shape) != hshape or history.dtype != dtype):
        raise ValueError("history must be %s %s" % (hshape, dtype))
    for name, t, shape in (("x", x, lead + (x_dim,)), ("B", B, lead + (bc_dim,)),
                           ("C", C, lead + (bc_dim,)), ("history_out", history_out, hshape)):
        if t is not None and (tuple(t.shape) != shape or t.dtype != dtype
                              or not t.is_contiguous()):
            raise ValueError("%s must be a contiguous %s %s tensor" % (name, shape, dtype))
    prob = ConvProblem(batch, L, num_seqs, x_dim, bc_dim, K, in_stride, _DTYPES[dtype], 0)
    context, handle = _stream_of(dev, stream)
    # copies and outputs are made on the stream the kernel runs on (see step())
    with context:
        cu = (cu_seqlens.to(device=dev, dtype=torch.int32).contiguous() if cu_seqlens is not None
              else None)
        weight = weight.contiguous()
        bias = bias.contiguous() if bias is not None else None
        history = history.contiguous() if history is not None else None
        if x is None:
            x = torch.empty(lead + (x_dim,), device=dev, dtype=dtype)
        if B is None:
            B = torch.empty(lead + (bc_dim,), device=dev, dtype=dtype)
        if C is None:
            C = torch.empty(lead + (bc_dim,), device=dev, dtype=dtype)
        if history_out is None and want_history:
            history_out = torch.empty(hshape, device=dev, dtype=dtype)
        tensors = (_addr(weight), _addr(bias), _addr(history), _addr(cu), _addr(x), _addr(B),
                   _addr(C), _addr(history_out), handle)
        if kept is not None:
            _check(load().ssd_conv1d_silu_checkpoint(prob, None, kept.arg(), *tensors),
                   "ssd_conv1d_silu_checkpoint")
        elif checkpoint is not False:
            save = _checkpoint_out(checkpoint, tuple(xbc.shape), dtype, dev)
            _check(load().ssd_conv1d_silu_checkpoint(prob, xbc.data_ptr(), save.arg(), *tensors),
                   "ssd_conv1d_silu_checkpoint")
            return x, B, C, history_out, save
        else:
            _check(load().ssd_conv1d_silu(prob, xbc.data_ptr(), *tensors), "ssd_conv1d_silu")
    return x, B, C, history_out


class BackwardPlan:
    """A prepared ssd_backward call for one forward problem: the problem is
    validated and the gradient outputs and workspace allocated once; :meth:`run`
    only enqueues the kernels.

    Takes the forward inputs (as for :class:`Plan`; bf16) and dL/dy, and
    optionally dL/d(final state); the states are recomputed. Returns from :meth:`run` a dict
    with dx, ddt, dA, dB, dC, dD, dinitial_state (dD without D is the gradient
    at D = 0; dinitial_state without an initial state the gradient at zero).
    """

    def __init__(self, x, dt, A, B, C, D, initial_state, dy, dfinal_state=None,
                 chunk_size=256, cu_seqlens=None, *, check_cu_seqlens=True):
        if x.dim() != 4:
            raise ValueError("x must be (batch, seqlen, nheads, headdim)")
        batch, L, H, P = x.shape
        G, N = B.shape[2], B.shape[3]
        dev = x.device
        _same_device(dev, dt=dt, A=A, B=B, C=C, D=D, initial_state=initial_state, dy=dy,
                     dfinal_state=dfinal_state)
        _on_gpu(dev)
        if x.dtype != torch.bfloat16:
            raise ValueError("the backward pass takes bfloat16 problems")
        for name, t, shape in (("dt", dt, (batch, L, H)), ("B", B, (batch, L, G, N)),
                               ("C", C, (batch, L, G, N)), ("dy", dy, tuple(x.shape))):
            if tuple(t.shape) != shape or t.dtype != x.dtype or t.device != dev:
                raise ValueError("%s must be %s %s on %s" % (name, shape, x.dtype, dev))
        if tuple(A.shape) != (H,) or A.dtype != torch.float32:
            raise ValueError("A must be (H,) float32")
        if D is not None and (tuple(D.shape) != (H,) or D.dtype != torch.float32):
            raise ValueError("D must be (H,) float32")
        num_seqs = 0
        if cu_seqlens is not None:
            if batch != 1:
                raise ValueError("cu_seqlens needs batch == 1")
            num_seqs = int(cu_seqlens.numel()) - 1
        nstate = num_seqs if num_seqs else batch
        for name, t in (("initial_state", initial_state), ("dfinal_state", dfinal_state)):
            if t is not None and (tuple(t.shape) != (nstate, H, P, N) or t.dtype != torch.float32):
                raise ValueError("%s must be (%d, %d, %d, %d) float32" % (name, nstate, H, P, N))
        self.prob = make_problem(batch, L, H, P, N, G, chunk_size, num_seqs, SSD_DTYPE_BF16, 0)
        validate(self.prob)
        self.cu = None
        if cu_seqlens is not None:
            if check_cu_seqlens or cu_seqlens.device.type == "cpu":
                validate_cu_seqlens(self.prob, cu_seqlens.detach().cpu())
            self.cu = cu_seqlens.to(device=dev, dtype=torch.int32).contiguous()
        n = ctypes.c_size_t(0)
        _check(load().ssd_backward_workspace_size(ctypes.byref(self.prob), ctypes.byref(n)),
               "ssd_backward_workspace_size")
        self.inputs = [t.contiguous() if t is not None else None
                       for t in (x, dt, A, B, C, D, initial_state, dy, dfinal_state)]
        self.grads = dict(
            dx=torch.empty_like(x), ddt=torch.empty_like(dt),
            dA=torch.empty(H, device=dev, dtype=torch.float32),
            dB=torch.empty_like(B), dC=torch.empty_like(C),
            dD=torch.empty(H, device=dev, dtype=torch.float32),
            dinitial_state=torch.empty((nstate, H, P, N), device=dev, dtype=torch.float32))
        self.workspace = torch.empty(max(n.value, 256), device=dev, dtype=torch.uint8)
        self.tokens = batch * L

    def _args(self, stream):
        x, dt, A, B, C, D, h0, dy, dhT = self.inputs
        g = self.grads
        return [ctypes.byref(self.prob), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                _ptr(h0), _ptr(self.cu), _ptr(dy), _ptr(dhT), _ptr(g["dx"]),
                _ptr(g["ddt"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]),
                _ptr(g["dinitial_state"]), _ptr(self.workspace),
                ctypes.c_size_t(self.workspace.numel()), ctypes.c_void_p(stream.cuda_stream)]

    def run(self, stream=None):
        """Enqueue one backward pass on ``stream`` (default: torch's current)."""
        if stream is None:
            stream = torch.cuda.current_stream(self.workspace.device)
        _check(load().ssd_backward(*self._args(stream)), "ssd_backward")
        return self.grads

    def run_timed(self, iterations: int, stream=None) -> StageTimes:
        """``iterations`` passes with a HIP event after every kernel; waits for
        them and returns the per-kernel times (see ssd_backward_timed)."""
        if stream is None:
            stream = torch.cuda.current_stream(self.workspace.device)
        times = StageTimes()
        _check(load().ssd_backward_timed(*self._args(stream), int(iterations),
                                         ctypes.byref(times)), "ssd_backward_timed")
        return times


def backward(x, dt, A, B, C, D, initial_state, dy, dfinal_state=None, chunk_size=256,
             cu_seqlens=None):
    """SSD backward pass (ssd_backward): a dict of gradients (see BackwardPlan)."""
    return BackwardPlan(x, dt, A, B, C, D, initial_state, dy, dfinal_state, chunk_size,
                        cu_seqlens).run()


def conv1d_silu_backward(xbc, weight, bias, dx, dB, dC, history=None, cu_seqlens=None, *,
                         dhistory_out=None, dxbc=None, check_cu_seqlens=True, stream=None):
    """The convolution front backwards (ssd_conv1d_silu_backward): a dict with
    dxbc, dweight, dbias and dhistory (None without a history).

    xbc, weight, bias, history and cu_seqlens as given to :func:`conv1d_silu`
    (xbc may be a :class:`Checkpoint` of it). dx, dB and dC are the gradients
    of its outputs, as :func:`backward` returns them (packed, with its batch
    axis of 1) or with their channels flattened; dhistory_out that of history_out, or None. dxbc (optional
    output, shaped like xbc) may be a slice of wider rows and must not overlap
    the inputs. dbias without a bias is the gradient at zero.
    """
    kept = xbc if isinstance(xbc, Checkpoint) else None
    dtype = xbc.dtype
    u = kept.q if kept is not None else xbc
    dev = u.device
    _same_device(dev, weight=weight, bias=bias, dx=dx, dB=dB, dC=dC, history=history,
                 dhistory_out=dhistory_out, dxbc=dxbc)
    _on_gpu(dev)
    if dtype not in _DTYPES:
        raise ValueError("xbc must be bfloat16 or float32")
    packed = cu_seqlens is not None
    if u.dim() != (2 if packed else 3):
        raise ValueError("packed xbc must be (tokens, channels)" if packed else
                         "dense xbc must be (batch, seqlen, channels)")
    lead, ch = tuple(u.shape[:-1]), int(u.shape[-1])
    if packed:
        batch, L, num_seqs = 1, lead[0], int(cu_seqlens.numel()) - 1
        nseq = num_seqs
        if num_seqs < 1:
            raise ValueError("cu_seqlens must hold at least two offsets")
        if check_cu_seqlens or cu_seqlens.device.type == "cpu":
            _check_offsets(cu_seqlens, L)
    else:
        (batch, L), num_seqs = lead, 0
        nseq = batch
    if batch * L >= _MOST_TOKENS or nseq >= _MOST_TOKENS:
        raise ValueError("%d tokens in %d sequences are more than one call takes"
                         % (batch * L, nseq))
    x_dim, bc_dim, also = (_channels_after(lead, name, t, dtype)
                           for name, t in (("dx", dx), ("dB", dB), ("dC", dC)))
    if also != bc_dim or x_dim + 2 * bc_dim != ch:
        raise ValueError("dx, dB, dC have %d, %d, %d channels, but xbc has %d"
                         % (x_dim, bc_dim, also, ch))
    K = weight.shape[1] if weight.dim() == 2 else 0
    if weight.shape != (ch, K) or weight.dtype != torch.float32:
        raise ValueError("weight must be (%d, K) float32" % ch)
    if bias is not None and (bias.shape != (ch,) or bias.dtype != torch.float32):
        raise ValueError("bias must be (%d,) float32" % ch)
    hshape = (nseq, K - 1, ch)
    for name, t in (("history", history), ("dhistory_out", dhistory_out)):
        if t is not None and (t.shape != hshape or t.dtype != dtype):
            raise ValueError("%s must be %s %s" % (name, hshape, dtype))
    if dxbc is not None and (dxbc.shape != u.shape or dxbc.dtype != dtype):
        raise ValueError("dxbc must be %s %s" % (lead + (ch,), dtype))
    context, handle = _stream_of(dev, stream)
    # copies, outputs and the workspace are made on the stream the kernels run on
    with context:
        cu_dev = cu_seqlens.to(device=dev, dtype=torch.int32).contiguous() if packed else None
        if dxbc is None:
            dxbc, out_stride = dx.new_empty(lead + (ch,)), ch
        else:
            out_stride = _stride_of_out(dxbc, "dxbc")
        in_stride = ch
        if kept is None:
            u, in_stride = _rows_in(u)
        if max(in_stride, out_stride) >= 1 << 31:
            raise ValueError("the rows of xbc or dxbc are too far apart")
        dx, dB, dC = _dense(dx), _dense(dB), _dense(dC)
        history, dhistory_out = _dense(history), _dense(dhistory_out)
        weight = weight.contiguous()
        bias = bias.contiguous() if bias is not None else None
        dweight, dbias = weight.new_empty((ch, K)), weight.new_empty(ch)
        dhistory = dx.new_empty(hshape) if history is not None else None
        sizes = (batch, L, num_seqs, x_dim, bc_dim, K, in_stride, _DTYPES[dtype], 0)
        prob, n = _conv_backward_bytes(*sizes)
        ws = torch.empty(n, device=dev, dtype=torch.uint8) if n else None
        _check(load().ssd_conv1d_silu_backward(
            prob, None if kept is not None else u.data_ptr(),
            kept.arg() if kept is not None else None, weight.data_ptr(), _addr(bias),
            _addr(history), _addr(cu_dev), dx.data_ptr(), dB.data_ptr(), dC.data_ptr(),
            _addr(dhistory_out), dxbc.data_ptr(), out_stride, dweight.data_ptr(),
            dbias.data_ptr(), _addr(dhistory), _addr(ws), n, handle),
            "ssd_conv1d_silu_backward")
    return dict(dxbc=dxbc, dweight=dweight, dbias=dbias, dhistory=dhistory)


@functools.lru_cache(maxsize=256)
def _conv_backward_bytes(*sizes):
    """The problem (read only) and workspace bytes of a front's backward pass,
    by its sizes."""
    prob, n = ConvProblem(*sizes), ctypes.c_size_t(0)
    _check(load().ssd_conv1d_silu_backward_workspace_size(prob, ctypes.byref(n)),
           "ssd_conv1d_silu_backward_workspace_size")
    return prob, n.value


def _channels_after(lead, name, t, dtype):
    """Channels of a gradient shaped ``lead`` + one or more axes of them; packed
    (``lead`` the tokens alone), a batch axis of 1 may stand before the tokens."""
    shape, n = t.shape, len(lead)
    if n == 1 and len(shape) > 2 and shape[0] == 1 and shape[1] == lead[0]:
        shape = shape[1:]
    if len(shape) <= n or shape[:n] != lead or t.dtype != dtype:
        raise ValueError("%s must be %s + channels, %s" % (name, lead, dtype))
    return shape[n] if len(shape) == n + 1 else shape[n:].numel()


@functools.lru_cache(maxsize=256)
def _norm_backward_bytes(*sizes):
    """Workspace bytes of a norm's backward pass, by its sizes."""
    n = ctypes.c_size_t(0)
    _check(load().ssd_group_norm_silu_backward_workspace_size(NormProblem(0, 0, 0, 0, 0, *sizes),
                                                              ctypes.byref(n)),
           "ssd_group_norm_silu_backward_workspace_size")
    return n.value


def _norm_sizes(x, groups, eps, center, norm_before_gate):
    """(tokens, channels, groups, dtype, flags, eps) of a NormProblem."""
    shape = x.shape
    channels = shape[-1] if len(shape) else 0
    if channels < 1 or x.dtype not in _DTYPES:
        raise ValueError("x must be bfloat16 or float32 with a channel axis")
    tokens = shape.numel() // channels
    if tokens >= _MOST_TOKENS:
        raise ValueError("%d tokens are more than one call takes" % tokens)
    if not 0 < groups <= channels:
        raise ValueError("groups (%d) must be between 1 and the channel count %d"
                         % (groups, channels))
    flags = (SSD_NORM_CENTER if center else 0) | (SSD_NORM_BEFORE_GATE if norm_before_gate else 0)
    return tokens, channels, groups, _DTYPES[x.dtype], flags, eps


def _norm_tensors(x, channels, like, weight, bias):
    """Checks of a norm's tensors: ``like`` (name -> tensor or None) are laid
    out as x, the parameters (channels,) float32; all on x's device. z is a
    Checkpoint where x is one, nothing else may be."""
    shape, dtype, dev = x.shape, x.dtype, x.device
    kept = isinstance(x, Checkpoint)
    for name, t in like.items():
        if t is not None:
            if t.device != dev or isinstance(t, Checkpoint):
                _same_device(dev, **{name: t.q if kept and name == "z" else t})
            if t.shape != shape or t.dtype != dtype:
                raise ValueError("%s must be %s %s" % (name, tuple(shape), dtype))
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            if isinstance(t, Checkpoint) or t.device != dev:
                _same_device(dev, **{name: t})
            if t.shape != (channels,) or t.dtype != torch.float32:
                raise ValueError("%s must be (%d,) float32" % (name, channels))
    _on_gpu(dev)


def _pair(checkpoint):
    """The caller's pair of Checkpoints to fill, of x and of z (or None)."""
    if not isinstance(checkpoint, (tuple, list)) or len(checkpoint) != 2:
        raise ValueError("checkpoint must be True, False or a pair of Checkpoints to fill")
    x, z = checkpoint
    if x is not True and x is z:
        raise ValueError("x and z need a Checkpoint each")
    return x, z


def group_norm_silu(x, weight=None, bias=None, z=None, *, groups=1, eps=1e-5, center=False,
                    norm_before_gate=False, checkpoint=False, out=None, stream=None):
    """Group norm with SiLU, channels last (ssd_group_norm_silu): the gate
    between the layer's output and the output projection. Returns ``out``.

    x (..., channels), bfloat16 or float32; z like x or None; weight, bias
    (channels,) float32 or None. Every token is normalised over ``groups``
    groups of consecutive channels (a multiple of 8 up to 16384 each), by its
    root mean square, or with ``center`` by its mean and standard deviation:
    norm(x * silu(z)) * weight + bias; with ``norm_before_gate``
    (norm(x) * weight + bias) * silu(z); without z silu(norm(x) * weight + bias).
    x, z and out may be slices of wider rows. With ``checkpoint=True`` x and z
    are also kept in 8 bits on the way: returns (out, x's Checkpoint, z's or
    None); a pair of Checkpoints is filled instead. Outputs must not overlap
    inputs.
    """
    if isinstance(x, Checkpoint):
        _refuse_checkpoint("x")
    sizes = _norm_sizes(x, groups, eps, center, norm_before_gate)
    dev, dtype, shape = x.device, x.dtype, x.shape
    _norm_tensors(x, sizes[1], {"z": z, "out": out}, weight, bias)
    if norm_before_gate and z is None:
        raise ValueError("norm_before_gate needs z")
    context, handle = _stream_of(dev, stream)
    # copies and outputs are made on the stream the kernel runs on
    with context:
        if out is None:
            out, out_stride = x.new_empty(shape), sizes[1]
        else:
            out_stride = _stride_of_out(out, "out")
        kx = kz = None
        if checkpoint is not False:
            gx, gz = (True, True) if checkpoint is True else _pair(checkpoint)
            kx = _checkpoint_out(gx, tuple(shape), dtype, dev)
            kz = _checkpoint_out(gz, tuple(shape), dtype, dev) if z is not None else None
        x, x_stride = _rows_in(x)
        z, z_stride = _rows_in(z) if z is not None else (None, 0)
        weight = weight.contiguous() if weight is not None else None
        bias = bias.contiguous() if bias is not None else None
        _check(load().ssd_group_norm_silu(
            NormProblem(x_stride, z_stride, out_stride, 0, 0, *sizes), x.data_ptr(), _addr(z),
            _addr(weight), _addr(bias), out.data_ptr(), kx.arg() if kx is not None else None,
            kz.arg() if kz is not None else None, handle), "ssd_group_norm_silu")
    return out if checkpoint is False else (out, kx, kz)


def group_norm_silu_backward(dout, x, weight=None, bias=None, z=None, *, groups=1, eps=1e-5,
                             center=False, norm_before_gate=False, dx=None, dz=None,
                             stream=None):
    """:func:`group_norm_silu` backwards (ssd_group_norm_silu_backward): a dict
    with dx, dz (None without z), dweight and dbias (each None without the
    parameter).

    The forward inputs and options as given there; x and z may both be
    :class:`Checkpoint` of the inputs. dout, and the optional outputs dx and
    dz, are shaped like x and may be slices of wider rows. Outputs must not
    overlap inputs.
    """
    kept = isinstance(x, Checkpoint)
    if z is not None and isinstance(z, Checkpoint) != kept:
        raise ValueError("x and z must both be tensors or both checkpoints")
    sizes = _norm_sizes(x, groups, eps, center, norm_before_gate)
    dev, dtype, shape = x.device, x.dtype, x.shape
    channels = sizes[1]
    _norm_tensors(x, channels, {"dout": dout, "z": z, "dx": dx, "dz": dz}, weight, bias)
    if dout is None:
        raise ValueError("dout is required")
    if z is None and (norm_before_gate or dz is not None):
        raise ValueError("norm_before_gate and dz need z")
    context, handle = _stream_of(dev, stream)
    # copies, outputs and the workspace are made on the stream the kernels run on
    with context:
        dx_stride = dz_stride = channels
        if dx is None:
            dx = dout.new_empty(shape)
        else:
            dx_stride = _stride_of_out(dx, "dx")
        if dz is not None:
            dz_stride = _stride_of_out(dz, "dz")
        elif z is not None:
            dz = dout.new_empty(shape)
        dout, out_stride = _rows_in(dout)
        x_stride = z_stride = 0
        if not kept:
            x, x_stride = _rows_in(x)
            z, z_stride = _rows_in(z) if z is not None else (None, 0)
        dweight = dbias = ws = None
        n = 0
        if weight is not None:
            weight = weight.contiguous()
            dweight = weight.new_empty(channels)
        if bias is not None:
            bias = bias.contiguous()
            dbias = bias.new_empty(channels)
        if weight is not None or bias is not None:
            n = _norm_backward_bytes(*sizes)
            ws = torch.empty(n, device=dev, dtype=torch.uint8) if n else None
        _check(load().ssd_group_norm_silu_backward(
            NormProblem(x_stride, z_stride, out_stride, dx_stride, dz_stride, *sizes),
            dout.data_ptr(), None if kept else x.data_ptr(), None if kept else _addr(z),
            x.arg() if kept else None, z.arg() if kept and z is not None else None,
            _addr(weight), _addr(bias), dx.data_ptr(), _addr(dz), _addr(dweight), _addr(dbias),
            _addr(ws), n, handle), "ssd_group_norm_silu_backward")
    return dict(dx=dx, dz=dz, dweight=dweight, dbias=dbias)
