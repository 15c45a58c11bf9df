"""Muon optimizer step for NVIDIA B200 (sm_100a).

Python binding of the C interface in include/muon.h.  This module only
marshals arguments: every step of the computation runs in libmuon.so's CUDA
kernels.  PyTorch provides device memory and streams.  There is no CPU
fallback: if libmuon.so is missing or no sm_100 device is present, the calls
raise.

    import newton_schulz_norm_b200 as muon
    muon.step(params, grads, bufs, lr=0.02)      # lists of 2-D fp32 CUDA tensors
"""
from __future__ import annotations

import array
import ctypes
import os
from typing import Sequence

import torch

__all__ = [
    "DEFAULT_COEFFS", "MuonError", "library", "step", "orthogonalize", "momentum_normalize",
    "gram", "poly", "xupdate", "status", "release", "workspace_bytes", "set_wait_limit_ns",
    "adamw_step", "AdamWGroup", "capture_step", "EXPORTS", "guard_check",
    "grad_norm", "clip_scale", "clip_grads", "GradGroup",
]

DEFAULT_COEFFS = (3.4445, -4.7750, 2.0315)
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmuon.so")

# Every symbol include/muon.h declares.
EXPORTS = ("muon_step", "muon_orthogonalize", "muon_momentum_normalize", "muon_gram", "muon_poly",
           "muon_xupdate", "muon_status", "muon_error_string", "muon_set_wait_limit_ns",
           "muon_workspace_bytes", "muon_release", "muon_version", "muon_profile_begin",
           "muon_profile_end", "muon_momentum_normalize_noalloc", "muon_adamw_step",
           "muon_step_mirrored", "muon_guard_check", "muon_grad_workspace_bytes", "muon_grad_norm",
           "muon_clip_grads", "muon_step_scaled", "muon_adamw_step_scaled",
           "muon_momentum_normalize_scaled")

PROFILE_KINDS = ("momentum_norm_cast", "gram", "poly", "xupdate", "xupdate_final", "apply", "adamw",
                 "ns_chain", "grad_norm", "grad_scale")

_STATUS = {0: "MUON_OK", -1: "MUON_ERR_INVALID_ARG", -2: "MUON_ERR_UNSUPPORTED",
           -3: "MUON_ERR_CUDA", -4: "MUON_ERR_NOMEM", -5: "MUON_ERR_TIMEOUT"}


class MuonError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {_STATUS.get(code, code)} ({code})")


_lib = None

_P = ctypes.c_void_p
_PP = ctypes.POINTER(ctypes.c_void_p)
_I64P = ctypes.POINTER(ctypes.c_int64)
_FP = ctypes.POINTER(ctypes.c_float)


def library() -> ctypes.CDLL:
    """Load libmuon.so (built in-tree by newton_schulz_norm_b200.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: run `python -m newton_schulz_norm_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    i, i64, f, u64, d = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_uint64, ctypes.c_double
    sig = {
        "muon_step": (i, [_PP, _PP, _PP, _I64P, i, f, f, i, i, _FP, _P]),
        "muon_orthogonalize": (i, [_P, _P, i, i64, i64, i, _FP, _P]),
        "muon_momentum_normalize": (i, [_PP, _PP, _PP, _I64P, _I64P, i, f, i, _P]),
        "muon_gram": (i, [_P, i64, _P, i64, i64, i64, _P]),
        "muon_poly": (i, [_P, i64, _P, i64, i64, f, f, _P]),
        "muon_xupdate": (i, [_P, i64, _P, i64, _P, i64, i64, i64, f, _P]),
        "muon_status": (i, [_P]),
        "muon_error_string": (ctypes.c_char_p, [i]),
        "muon_set_wait_limit_ns": (None, [u64]),
        "muon_workspace_bytes": (i64, [_I64P, i]),
        "muon_release": (None, []),
        "muon_version": (ctypes.c_char_p, []),
        "muon_profile_begin": (None, []),
        "muon_profile_end": (i, [ctypes.POINTER(ctypes.c_double), _I64P, i]),
        "muon_momentum_normalize_noalloc": (i, [_PP, _PP, _PP, _I64P, _I64P, i, f, i, _P, _P]),
        "muon_adamw_step": (i, [_PP, _PP, _PP, _PP, _I64P, _P, i, i64, d, d, d, d, d, _P]),
        "muon_step_mirrored": (i, [_PP, _PP, _PP, _I64P, i, f, f, i, i, _FP, _PP, i, _P]),
        "muon_guard_check": (i64, []),
        "muon_grad_workspace_bytes": (i64, [_P, _I64P, i]),
        "muon_grad_norm": (i, [_P, _P, _P, i, d, d, d, _P, _P, _P, i64, _P]),
        "muon_clip_grads": (i, [_P, _P, _P, i, _P, _P, d, d, d, _P, _P, _P, i64, _P]),
        "muon_step_scaled": (i, [_PP, _PP, _PP, _I64P, i, f, f, i, i, _FP, _PP, i, _P, _P]),
        "muon_adamw_step_scaled": (i, [_P, _P, _P, _P, _P, _P, i, i64, d, d, d, d, d, _P, _P]),
        "muon_momentum_normalize_scaled": (i, [_P, _P, _P, _P, _P, i, f, i, _P, _P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(code: int, what: str):
    if code != 0:
        raise MuonError(code, what)


def _raw_stream(device: int) -> int:
    """Handle of torch's current stream on a device."""
    return int(torch.cuda.current_stream(device).cuda_stream)


# The same without building a Stream object (0.1 instead of 3.2 us per call),
# where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _stream_ptr(stream) -> int:
    if stream is None:
        if torch.cuda.is_initialized():
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr_array(tensors) -> ctypes.Array:
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def _coeffs(coeffs):
    if coeffs is None:
        return None
    return (ctypes.c_float * 3)(*[float(c) for c in coeffs])


def _torch_stream(stream):
    """A torch stream for a stream argument (a stream object or a handle)."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    ptr = _stream_ptr(stream)
    return torch.cuda.ExternalStream(ptr) if ptr else torch.cuda.default_stream()


def _is_side(stream) -> bool:
    """Whether a stream argument names another stream than torch's current one."""
    return stream is not None and _stream_ptr(stream) != _stream_ptr(None)


def _scale_ptr(grad_scale, stream=None):
    """Device address of a gradient scale (a one-element fp32 CUDA tensor on
    the current device), or None.  Where ``stream`` is not torch's current one
    the allocator is told, so that a scale dropped after the call is not handed
    out again before the kernels there have read it."""
    if grad_scale is None:
        return None
    if not isinstance(grad_scale, torch.Tensor) or grad_scale.get_device() < 0 \
            or grad_scale.dtype is not torch.float32 or grad_scale.numel() != 1:
        raise ValueError("grad_scale: expected a float32 CUDA tensor of one element")
    if grad_scale.get_device() != torch.cuda.current_device():
        _check_device(grad_scale.get_device(), "grad_scale")
    if _is_side(stream):
        grad_scale.record_stream(_torch_stream(stream))
    return grad_scale.data_ptr()


def _check_device(index: int, name: str):
    if index != torch.cuda.current_device():
        raise ValueError(f"{name}: on cuda:{index}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _device_for(tensors):
    """Index of the current device, asked once for a list; None where the first
    of the list is no CUDA tensor, which the checks of the list then refuse."""
    t = next(iter(tensors), None)
    return torch.cuda.current_device() if isinstance(t, torch.Tensor) and t.is_cuda else None


def _check_mat(t: torch.Tensor, name: str, dtype=torch.float32, device: int | None = None):
    """``device``: index of the current device, where the caller has it.  A tensor
    in order is asked few things: for a list of many this takes longer than
    launching its kernels."""
    if isinstance(t, torch.Tensor) and t.ndim == 2 and t.dtype is dtype and t.get_device() == device \
            and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor) or t.ndim != 2:
        raise ValueError(f"{name}: expected a 2-D tensor")
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} CUDA tensor")
    if t.get_device() != (torch.cuda.current_device() if device is None else device):
        _check_device(t.get_device(), name)


def _refuse_vector(t, name: str):
    """Raises for a tensor that is not a contiguous fp32 one on the current device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous float32 CUDA tensor")
    _check_device(t.get_device(), name)


def _as_matrix(t: torch.Tensor) -> torch.Tensor:
    """View an N-D (N >= 3) tensor as (shape[0], prod(shape[1:])) -- a conv
    weight as its im2col matrix.  1-D tensors are not Muon parameters."""
    if t.dim() < 2:
        raise ValueError("Muon updates matrices; 1-D parameters belong to another optimizer")
    if t.dim() == 2:
        return t
    if not t.is_contiguous():
        raise ValueError("an N-D tensor must be contiguous to be updated through its matrix view")
    return t.view(t.shape[0], -1)   # a view: the in-place update reaches t


def step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
         bufs: Sequence[torch.Tensor], lr: float, beta: float = 0.95, nesterov: bool = True,
         ns_steps: int = 5, coeffs=DEFAULT_COEFFS, stream=None, reshape_nd: bool = False,
         mirrors=None, grad_scale: torch.Tensor | None = None) -> None:
    """One Muon step, in place on params and bufs (see include/muon.h).

    With reshape_nd, tensors of rank >= 3 (conv weights) are updated as their
    (shape[0], prod(shape[1:])) matrix view; they must be contiguous.

    mirrors: optional list of destinations, each a list with one entry per
    parameter (a tensor of the same shape, or a raw device address, e.g. of
    another GPU's copy); the last kernel writes every updated matrix to each
    of them as well (muon_step_mirrored).

    grad_scale: optional one-element fp32 CUDA tensor (clip_scale's) that
    multiplies every gradient on the way in; grads themselves stay as they are.
    """
    n = len(params)
    if len(grads) != n or len(bufs) != n:
        raise ValueError("params, grads and bufs must have the same length")
    if reshape_nd:
        params = [_as_matrix(t) for t in params]
        grads = [_as_matrix(t) for t in grads]
        bufs = [_as_matrix(t) for t in bufs]
    shapes = []
    device = _device_for(params)
    for p, g, b in zip(params, grads, bufs):
        for t, nm in ((p, "param"), (g, "grad"), (b, "buf")):
            _check_mat(t, nm, device=device)
        shape = p.shape
        if g.shape != shape or b.shape != shape:
            raise ValueError("param, grad and buf shapes differ")
        shapes += shape
    sh = (ctypes.c_int64 * len(shapes))(*shapes)
    if mirrors:
        flat = []
        for dests in mirrors:
            if len(dests) != n:
                raise ValueError("every mirror needs one destination per parameter")
            for t, p in zip(dests, params):
                if isinstance(t, torch.Tensor):
                    if t.shape != p.shape or t.dtype != torch.float32 or not t.is_contiguous():
                        raise ValueError("a mirror tensor must match its parameter (contiguous fp32)")
                    flat.append(t.data_ptr())
                else:
                    flat.append(int(t))
        mir = (ctypes.c_void_p * len(flat))(*flat)
    else:
        mir, mirrors = None, ()
    code = library().muon_step_scaled(
        _ptr_array(params), _ptr_array(grads), _ptr_array(bufs), sh, n, float(lr), float(beta),
        int(bool(nesterov)), int(ns_steps), _coeffs(coeffs), mir, len(mirrors),
        _scale_ptr(grad_scale, stream), _stream_ptr(stream))
    _check(code, "muon_step_mirrored" if mirrors else "muon_step")


def capture_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                 bufs: Sequence[torch.Tensor], lr: float, beta: float = 0.95,
                 nesterov: bool = True, ns_steps: int = 5, coeffs=DEFAULT_COEFFS,
                 reshape_nd: bool = False,
                 grad_scale: torch.Tensor | None = None) -> "torch.cuda.CUDAGraph":
    """Run one Muon step eagerly, then capture the next one in a CUDA graph.

    The first call for a set of shapes and parameter pointers builds the
    library's plan and tensor maps (allocation and host copies, which a
    capture cannot hold); that is why this function performs one real step
    before capturing.  Every ``replay()`` of the returned graph is one more
    step on the same tensors: write each step's gradients into ``grads`` in
    place before replaying.  The graph keeps the hyper-parameters it was
    captured with, but reads ``grad_scale`` (when given) anew each time: write
    each step's scale into that tensor before replaying, and keep it as long as
    the graph, like every other tensor of the step.  Launching nothing but
    kernels and one memset, a replay saves the host work and launch gaps of the
    eager call.
    """
    kw = dict(lr=lr, beta=beta, nesterov=nesterov, ns_steps=ns_steps, coeffs=coeffs,
              reshape_nd=reshape_nd, grad_scale=grad_scale)
    step(params, grads, bufs, **kw)
    torch.cuda.synchronize()
    _check(status(), "muon_step (before capture)")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(params, grads, bufs, **kw)
    return graph


def step_raw(param_ptrs, grad_ptrs, buf_ptrs, shapes, lr, beta=0.95, nesterov=True, ns_steps=5,
             coeffs=DEFAULT_COEFFS, stream=0) -> int:
    """muon_step on raw device pointers; returns the status code unchanged."""
    n = len(param_ptrs)
    arr = lambda xs: (ctypes.c_void_p * max(n, 1))(*xs)  # noqa: E731
    flat = [int(v) for s in shapes for v in s]
    sh = (ctypes.c_int64 * max(len(flat), 1))(*flat)
    return library().muon_step(arr(param_ptrs), arr(grad_ptrs), arr(buf_ptrs), sh, n, float(lr),
                               float(beta), int(bool(nesterov)), int(ns_steps), _coeffs(coeffs),
                               int(stream) if stream is not None else None)


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
               exp_avgs: Sequence[torch.Tensor], exp_avg_sqs: Sequence[torch.Tensor], step: int,
               lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 1e-2,
               decay: Sequence[bool] | None = None, stream=None,
               grad_scale: torch.Tensor | None = None) -> None:
    """One AdamW step, in place on params and both running averages (see
    include/muon.h).  Tensors: fp32, contiguous, on the GPU, any shape; the
    four lists match element by element.  ``decay[i]`` false puts tensor i in
    the no-decay group; ``decay=None`` decays all.  ``step`` counts from 1.
    ``grad_scale``: optional one-element fp32 CUDA tensor (clip_scale's) that
    multiplies every gradient on the way in."""
    n = len(params)
    if not (len(grads) == len(exp_avgs) == len(exp_avg_sqs) == n):
        raise ValueError("params, grads, exp_avgs and exp_avg_sqs must have the same length")
    if decay is not None and len(decay) != n:
        raise ValueError("decay must have one entry per tensor")
    numels = []
    device = _device_for(params)
    tensor, f32 = torch.Tensor, torch.float32
    for p, g, m, v in zip(params, grads, exp_avgs, exp_avg_sqs):
        for t, nm in ((p, "param"), (g, "grad"), (m, "exp_avg"), (v, "exp_avg_sq")):
            if not (isinstance(t, tensor) and t.dtype is f32 and t.get_device() == device and t.is_contiguous()):
                _refuse_vector(t, nm)
        shape = p.shape
        if g.shape != shape or m.shape != shape or v.shape != shape:
            raise ValueError("param, grad and average shapes differ")
        numels.append(p.numel())
    code = adamw_step_raw([t.data_ptr() for t in params], [t.data_ptr() for t in grads],
                          [t.data_ptr() for t in exp_avgs], [t.data_ptr() for t in exp_avg_sqs],
                          numels, step, lr, betas, eps, weight_decay, decay, _stream_ptr(stream),
                          _scale_ptr(grad_scale, stream))
    _check(code, "muon_adamw_step")


class AdamWGroup:
    """A fixed set of AdamW tensors, checked and marshalled once.

    ``adamw_step`` validates and packs every tensor on every call (200
    microseconds of host time for a hundred tensors); a training loop that
    steps the same tensors each time can build the argument arrays once and
    then call ``step(t)``, which only passes them on.  The tensors must stay
    allocated (and at the same addresses) for the group's lifetime.
    """

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                 exp_avgs: Sequence[torch.Tensor], exp_avg_sqs: Sequence[torch.Tensor],
                 lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 1e-2,
                 decay: Sequence[bool] | None = None):
        n = len(params)
        if not (len(grads) == len(exp_avgs) == len(exp_avg_sqs) == n):
            raise ValueError("params, grads, exp_avgs and exp_avg_sqs must have the same length")
        if decay is not None and len(decay) != n:
            raise ValueError("decay must have one entry per tensor")
        first = next(iter(params), None)
        self._device = first.get_device() if isinstance(first, torch.Tensor) else None
        for p, g, m, v in zip(params, grads, exp_avgs, exp_avg_sqs):
            for t, nm in ((p, "param"), (g, "grad"), (m, "exp_avg"), (v, "exp_avg_sq")):
                if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32 \
                        or not t.is_contiguous():
                    raise ValueError(f"{nm}: expected a contiguous float32 CUDA tensor")
                if t.get_device() != self._device:
                    raise ValueError("every tensor must be on one device")
            if g.shape != p.shape or m.shape != p.shape or v.shape != p.shape:
                raise ValueError("param, grad and average shapes differ")
        self._keep = (list(params), list(grads), list(exp_avgs), list(exp_avg_sqs))
        self._n = n
        arr = lambda ts: (ctypes.c_void_p * max(n, 1))(*[t.data_ptr() for t in ts])  # noqa: E731
        self._p, self._g, self._m, self._v = (arr(ts) for ts in self._keep)
        self._numels = (ctypes.c_int64 * max(n, 1))(*[p.numel() for p in params])
        self._decay = None if decay is None else \
            (ctypes.c_ubyte * max(n, 1))(*[1 if d else 0 for d in decay])
        self.lr, self.betas, self.eps, self.weight_decay = float(lr), tuple(betas), float(eps), \
            float(weight_decay)
        at = ctypes.addressof
        self._args = (at(self._p), at(self._g), at(self._m), at(self._v), at(self._numels),
                      None if self._decay is None else at(self._decay), n)

    def step(self, step: int, lr: float | None = None, stream=None,
             grad_scale: torch.Tensor | None = None) -> None:
        """One AdamW step (t = ``step``, from 1) on the group's tensors;
        ``grad_scale`` as for adamw_step."""
        if self._device is not None and torch.cuda.current_device() != self._device:
            _check_device(self._device, "params")
        code = library().muon_adamw_step_scaled(
            *self._args, int(step), self.lr if lr is None else float(lr), float(self.betas[0]),
            float(self.betas[1]), self.eps, self.weight_decay, _scale_ptr(grad_scale, stream),
            _stream_ptr(stream))
        _check(code, "muon_adamw_step")


def adamw_step_raw(param_ptrs, grad_ptrs, avg_ptrs, sq_ptrs, numels, step, lr, betas=(0.9, 0.999),
                   eps=1e-8, weight_decay=1e-2, decay=None, stream=0, grad_scale=None) -> int:
    """muon_adamw_step on raw device pointers (grad_scale too); returns the status code unchanged."""
    n = len(param_ptrs)
    arr = lambda xs: (ctypes.c_void_p * max(n, 1))(*xs)  # noqa: E731
    ne = (ctypes.c_int64 * max(n, 1))(*[int(x) for x in numels])
    dm = None if decay is None else (ctypes.c_ubyte * max(n, 1))(*[1 if d else 0 for d in decay])
    return library().muon_adamw_step_scaled(
        arr(param_ptrs), arr(grad_ptrs), arr(avg_ptrs), arr(sq_ptrs), ne,
        ctypes.cast(dm, ctypes.c_void_p) if dm is not None else None, n, int(step), float(lr),
        float(betas[0]), float(betas[1]), float(eps), float(weight_decay), grad_scale,
        int(stream) if stream is not None else None)


_INF = float("inf")
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class GradGroup:
    """A fixed set of gradients for the norm and for clipping, checked and
    marshalled once (AdamWGroup does the same for its step).

    ``grads``: contiguous CUDA tensors of any shape on one device; float32,
    bfloat16 and float16 may be mixed, empty ones are skipped.  They must stay
    allocated at the same addresses for the group's lifetime; their values are
    read anew by every call.  ``out``: optional tensors of the same shapes, of
    any of the three types, that ``clip`` writes instead of ``grads`` (bf16
    gradients into the fp32 ones that the steps take, for instance); an entry
    may be the gradient itself, none may overlap anything else.

    Nothing is recorded for autograd: norms and scales are detached, whatever
    the tensors require.

    Every call takes its workspace and its results from torch's allocator on
    the call's stream, so calls on several streams and captures in several
    graphs do not disturb one another.  The library's first call on a device
    allocates; make it before any capture.
    """

    def __init__(self, grads: Sequence[torch.Tensor], out: Sequence[torch.Tensor] | None = None):
        n = len(grads)
        if out is not None and len(out) != n:
            raise ValueError("grads and out must have the same length")
        self._device = None
        for ts, nm in ((grads, "grad"), (out or (), "out")):
            for t in ts:
                if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _DTYPES \
                        or not t.is_contiguous():
                    raise ValueError(f"{nm}: expected a contiguous float32, bfloat16 or float16 CUDA tensor")
                if self._device is None:
                    self._device = t.device.index
                elif t.device.index != self._device:
                    raise ValueError("every tensor must be on one device")
        if out is not None and any(o.shape != g.shape for o, g in zip(out, grads)):
            raise ValueError("grad and out shapes differ")
        self._keep = (list(grads), None if out is None else list(out))
        self._n = n
        arr = lambda ts: (ctypes.c_void_p * max(n, 1))(*[t.data_ptr() for t in ts])  # noqa: E731
        kinds = lambda ts: (ctypes.c_ubyte * max(n, 1))(*[_DTYPES[t.dtype] for t in ts])  # noqa: E731
        self._g, self._gt = arr(grads), kinds(grads)
        self._o, self._ot = (self._g, self._gt) if out is None else (arr(out), kinds(out))
        self._numels = (ctypes.c_int64 * max(n, 1))(*[t.numel() for t in grads])
        self._bytes = int(library().muon_grad_workspace_bytes(self._gt, self._numels, n))
        if self._bytes < 0:
            raise ValueError("a gradient is too large")
        self._clippable = self._disjoint(grads, grads if out is None else out)
        if self._device is None:
            self._device = torch.cuda.current_device()
        # what the calls' results and workspaces are made like
        device = torch.device("cuda", self._device)
        self._result = torch.empty((), dtype=torch.float32, device=device)
        self._work = torch.empty(self._bytes, dtype=torch.uint8, device=device) if self._bytes else None
        at = ctypes.addressof
        self._args = (at(self._g), at(self._gt), at(self._numels), n, None, None)
        self._clip_args = self._args[:4] + (at(self._o), at(self._ot))

    @staticmethod
    def _disjoint(grads, outs) -> bool:
        """Whether no output overlaps another output, or a gradient other
        than its own (of the same type, at the same address)."""
        spans = []
        for i, (g, o) in enumerate(zip(grads, outs)):
            if o.numel() == 0:
                continue
            a, b = o.data_ptr(), g.data_ptr()
            spans.append((a, a + o.numel() * o.element_size(), True))
            if a != b or o.dtype != g.dtype:
                spans.append((b, b + g.numel() * g.element_size(), False))
        spans.sort()
        ends = {True: 0, False: 0}
        for a, e, written in spans:
            if a < ends[True] or (written and a < ends[False]):
                return False
            ends[written] = max(ends[written], e)
        return True

    def _call(self, args, p, max_norm, eps, with_scale, stream):
        if torch.cuda.current_device() != self._device:
            _check_device(self._device, "grads")
        if _is_side(stream):
            reader = torch.cuda.current_stream()
            with torch.cuda.stream(_torch_stream(stream)):   # the allocations below belong to that stream
                got = self._call(args, p, max_norm, eps, with_scale, None)
            for t in got if with_scale else (got,):
                t.record_stream(reader)
            return got
        norm = torch.empty_like(self._result)
        scale = torch.empty_like(self._result) if with_scale else None
        work = None if self._work is None else torch.empty_like(self._work)
        code = library().muon_clip_grads(
            *args, p, max_norm, eps, norm.data_ptr(), None if scale is None else scale.data_ptr(),
            None if work is None else work.data_ptr(), self._bytes, _raw_stream(self._device))
        if code:
            raise MuonError(code, "muon_grad_norm" if args is self._args else "muon_clip_grads")
        return (norm, scale) if with_scale else norm

    def norm(self, norm_type: float = 2.0, stream=None) -> torch.Tensor:
        """The norm over every gradient of the group, as a 0-d fp32 tensor.
        ``norm_type``: 1, 2 or inf (the largest magnitude)."""
        return self._call(self._args, float(norm_type), _INF, 0.0, False, stream)

    def clip_scale(self, max_norm: float, norm_type: float = 2.0, eps: float = 1e-6, stream=None):
        """(norm, scale): the norm, and min(1, max_norm / (norm + eps)) to be
        passed to the steps as ``grad_scale``.  Both 0-d fp32 tensors."""
        return self._call(self._args, float(norm_type), float(max_norm), float(eps), True, stream)

    def clip(self, max_norm: float, norm_type: float = 2.0, eps: float = 1e-6, stream=None) -> torch.Tensor:
        """Multiplies every gradient by min(1, max_norm / (norm + eps)), in
        place or into ``out``, and returns the norm they had."""
        if not self._clippable:
            raise ValueError("tensors that clip writes must not overlap other tensors of the group")
        return self._call(self._clip_args, float(norm_type), float(max_norm), float(eps), False, stream)


def grad_norm(grads: Sequence[torch.Tensor], norm_type: float = 2.0, stream=None) -> torch.Tensor:
    """The norm over every gradient of the list, as a 0-d fp32 tensor
    (GradGroup.norm; a loop over the same tensors keeps a GradGroup)."""
    return GradGroup(grads).norm(norm_type, stream)


def clip_scale(grads: Sequence[torch.Tensor], max_norm: float, norm_type: float = 2.0,
               eps: float = 1e-6, stream=None):
    """(norm, scale) of the list, the scale for the steps' ``grad_scale``:
    the steps then take clipped gradients without a pass that writes them."""
    return GradGroup(grads).clip_scale(max_norm, norm_type, eps, stream)


def clip_grads(grads: Sequence[torch.Tensor], max_norm: float, norm_type: float = 2.0,
               eps: float = 1e-6, out: Sequence[torch.Tensor] | None = None, stream=None) -> torch.Tensor:
    """Clip the list to ``max_norm``, in place or into ``out`` (same shapes,
    any of the three types), and return the norm it had."""
    return GradGroup(grads, out).clip(max_norm, norm_type, eps, stream)


def orthogonalize(x: torch.Tensor, ns_steps: int = 5, coeffs=DEFAULT_COEFFS,
                  out_dtype=torch.float32, out: torch.Tensor | None = None, stream=None):
    """Newton-Schulz orthogonalisation of one fp32 matrix (normalised first)."""
    _check_mat(x, "x")
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    _check_mat(out, "out", out.dtype)
    if out.dtype not in (torch.float32, torch.bfloat16) or out.shape != x.shape:
        raise ValueError("out must be fp32 or bf16 with the shape of x")
    code = library().muon_orthogonalize(x.data_ptr(), out.data_ptr(), int(out.dtype == torch.bfloat16),
                                        x.shape[0], x.shape[1], int(ns_steps), _coeffs(coeffs),
                                        _stream_ptr(stream))
    _check(code, "muon_orthogonalize")
    return out


def _ld8(n: int) -> int:
    return (n + 7) // 8 * 8


def momentum_normalize(grads, bufs, beta=0.95, nesterov=True, stream=None, grad_scale=None):
    """The fused first kernel alone; returns oriented bf16 X0 views (m x n).
    ``grad_scale`` as for step."""
    n = len(grads)
    if len(bufs) != n:
        raise ValueError("grads and bufs must have the same length")
    if _is_side(stream):
        _scale_ptr(grad_scale, stream)
        reader = torch.cuda.current_stream()
        with torch.cuda.stream(_torch_stream(stream)):   # the X0s belong to that stream
            outs = momentum_normalize(grads, bufs, beta, nesterov, None, grad_scale)
        for x in outs:
            x.record_stream(reader)
        return outs
    device = _device_for(grads)
    # One pass with few Python calls a matrix: for many small matrices this loop
    # takes longer than the kernel (array is quicker than ctypes here).
    tensor, f32, bf16, empty = torch.Tensor, torch.float32, torch.bfloat16, torch.empty_strided
    ptrs, lds, shapes, outs = [], [], [], []
    for g, b in zip(grads, bufs):
        shape = g.shape if isinstance(g, tensor) else ()
        if not (isinstance(b, tensor) and len(shape) == 2 and b.shape == shape and g.dtype is f32
                and b.dtype is f32 and g.get_device() == device and b.get_device() == device
                and g.is_contiguous() and b.is_contiguous()):
            _check_mat(g, "grad", device=device)
            _check_mat(b, "buf", device=device)
            raise ValueError("grad and buf shapes differ")
        r, c = shape
        m, nn = (r, c) if r <= c else (c, r)
        ld = (nn + 7) // 8 * 8
        # rows of ld elements, as a view of their first nn
        x = empty((m, nn), (ld, 1), dtype=bf16, device=g.device)
        outs.append(x)
        ptrs += (g.data_ptr(), b.data_ptr(), x.data_ptr())
        lds.append(ld)
        shapes += shape
    host = [array.array("q", v) for v in (ptrs[0::3], ptrs[1::3], ptrs[2::3], lds, shapes)]
    code = library().muon_momentum_normalize_scaled(
        *(a.buffer_info()[0] for a in host), n, float(beta), int(bool(nesterov)),
        _scale_ptr(grad_scale), _stream_ptr(stream))
    _check(code, "muon_momentum_normalize")
    return outs


def _bf16_padded(x: torch.Tensor) -> torch.Tensor:
    """Copy into a bf16 buffer whose row pitch is a multiple of 8 elements."""
    m, n = x.shape
    buf = torch.zeros((m, _ld8(n)), dtype=torch.bfloat16, device=x.device)
    buf[:, :n] = x
    return buf


def gram(x: torch.Tensor) -> torch.Tensor:
    """A = bf16(X X^T) for a bf16 m x n X (on the current stream)."""
    stream = None
    m, n = x.shape
    xp = _bf16_padded(x)
    a = torch.empty((m, _ld8(m)), dtype=torch.bfloat16, device=x.device)
    code = library().muon_gram(xp.data_ptr(), xp.shape[1], a.data_ptr(), a.shape[1], m, n,
                               _stream_ptr(stream))
    _check(code, "muon_gram")
    return a[:, :m]


def poly(a: torch.Tensor, cb: float, cc: float) -> torch.Tensor:
    """B = bf16(cb*A + cc*A A) for a symmetric bf16 m x m A (current stream)."""
    stream = None
    m = a.shape[0]
    ap = _bf16_padded(a)
    b = torch.empty((m, _ld8(m)), dtype=torch.bfloat16, device=a.device)
    code = library().muon_poly(ap.data_ptr(), ap.shape[1], b.data_ptr(), b.shape[1], m, float(cb),
                               float(cc), _stream_ptr(stream))
    _check(code, "muon_poly")
    return b[:, :m]


def xupdate(b: torch.Tensor, x: torch.Tensor, ca: float) -> torch.Tensor:
    """X' = bf16(ca*X + B X) for bf16 B (m x m) and X (m x n) (current stream)."""
    stream = None
    m, n = x.shape
    bp = _bf16_padded(b)
    xp = _bf16_padded(x)
    out = torch.empty((m, _ld8(n)), dtype=torch.bfloat16, device=x.device)
    code = library().muon_xupdate(bp.data_ptr(), bp.shape[1], xp.data_ptr(), xp.shape[1],
                                  out.data_ptr(), out.shape[1], m, n, float(ca), _stream_ptr(stream))
    _check(code, "muon_xupdate")
    return out[:, :n]


def status(stream=None) -> int:
    """Synchronise and return (and clear) the device-side status code."""
    return library().muon_status(_stream_ptr(stream))


def guard_check() -> int:
    """Synchronise and return how many guard-band bytes around the library's
    scratch regions were overwritten (0: no kernel wrote out of bounds)."""
    return int(library().muon_guard_check())


def release() -> None:
    library().muon_release()


def set_wait_limit_ns(ns: int) -> None:
    library().muon_set_wait_limit_ns(int(ns))


def workspace_bytes(shapes) -> int:
    flat = [int(v) for s in shapes for v in s]
    return int(library().muon_workspace_bytes((ctypes.c_int64 * max(len(flat), 1))(*flat), len(shapes)))


def version() -> str:
    return library().muon_version().decode()


def profile_begin() -> None:
    """Start bracketing every launch of the library with CUDA events."""
    library().muon_profile_begin()


def profile_end() -> dict:
    """Stop, synchronise, and return {kind: (total_ms, launches)}."""
    k = len(PROFILE_KINDS)
    ms = (ctypes.c_double * k)()
    n = (ctypes.c_int64 * k)()
    code = library().muon_profile_end(ms, n, k)
    if code < 0:
        raise MuonError(code, "muon_profile_end")
    return {PROFILE_KINDS[i]: (float(ms[i]), int(n[i])) for i in range(k)}


def momentum_normalize_noalloc(grads, bufs, x0s, beta=0.95, nesterov=True, dev_status=None,
                               stream=None) -> int:
    """The fused first kernel through the allocation-free entry point.

    For callers that must not allocate device memory while stepping: the
    library's scratch is a fixed array compiled into it.  ``x0s`` are
    caller-allocated bf16 buffers (min(r,c) x ld, ld % 8 == 0, ld >= max(r,c));
    ``dev_status`` an optional int32 CUDA tensor of one element that receives
    a device-side timeout.  Returns the status code (0 on success).
    """
    n = len(grads)
    shapes = [v for g in grads for v in g.shape]
    lds = [x.shape[1] for x in x0s]
    return library().muon_momentum_normalize_noalloc(
        _ptr_array(grads), _ptr_array(bufs), _ptr_array(x0s), (ctypes.c_int64 * max(n, 1))(*lds),
        (ctypes.c_int64 * max(len(shapes), 1))(*shapes), n, float(beta), int(bool(nesterov)),
        None if dev_status is None else dev_status.data_ptr(), _stream_ptr(stream))
