"""Thin Python binding of libmuon.so, the GB300 (sm_103a) Muon optimizer step.

Every function here has the name of the C entry point it calls (include/muon.h)
and only marshals arguments: torch tensors become device pointers and
``cudaStream_t`` handles; every step of the method runs in the library's
kernels.  PyTorch provides device memory (the workspace, the caller's tensors)
and streams.  There is no fallback: libmuon.so is loaded on first use and a
missing library raises ImportError there.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import os
import threading
from ctypes import POINTER, byref, c_char_p, c_float, c_int32, c_int64, c_size_t, c_void_p
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmuon.so")
# the same library with the device range checks of the debug build (use_debug_library)
LIB_PATH_DEBUG = os.path.join(_HERE, "libmuon_debug.so")

# status codes, dtypes and enums of include/muon.h
MUON_OK = 0
MUON_WARN_NONFINITE = 1
MUON_ERR_INVALID = -1
MUON_ERR_NOT_PINNED = -2
MUON_ERR_NO_WORKSPACE = -3
MUON_ERR_CUDA = -4
MUON_ERR_TIMEOUT = -5
MUON_ERR_UNSUPPORTED = -6
MUON_ERR_DEVICE = -7
MUON_DTYPE_F32 = 0
MUON_DTYPE_BF16 = 1
MUON_NS_BF16 = 0
MUON_NS_TF32X3 = 1
MUON_MOMENTUM_EMA = 0
MUON_MOMENTUM_SGD = 1
MUON_NS_KERNEL_AUTO = 0
MUON_NS_KERNEL_GEMM = 1
MUON_NS_METHOD_STANDARD = 0
MUON_NS_METHOD_GRAM = 1
MUON_MAX_NS_STEPS = 16
MUON_NONFINITE_KEEP = 0
MUON_NONFINITE_ZERO = 1
MUON_REDUCE_TOKEN_MEAN = 0
MUON_REDUCE_SEQUENCE_MEAN = 1
MUON_REDUCE_SUM = 2


class muon_shape(ctypes.Structure):
    _fields_ = [("rows", c_int64), ("cols", c_int64), ("count", c_int64), ("stride_elems", c_int64)]


class muon_config(ctypes.Structure):
    _fields_ = [("ns_a", c_float), ("ns_b", c_float), ("ns_c", c_float), ("eps", c_float),
                ("ns_precision", c_int32), ("momentum_form", c_int32), ("grad_dtype", c_int32),
                ("param_dtype", c_int32), ("max_inflight", c_int32), ("skip_nonfinite", c_int32),
                ("timing", c_int32), ("offload", c_int32), ("ns_kernel", c_int32),
                ("offload_zero_copy", c_int32), ("ns_momentum_fused", c_int32), ("ns_method", c_int32),
                ("reserved", c_int32 * 2)]


class muon_plan_info(ctypes.Structure):
    _fields_ = [("n_tensors", c_int64), ("n_matrices", c_int64), ("n_groups", c_int64),
                ("n_buckets", c_int64), ("max_bucket_matrices", c_int64),
                ("max_bucket_bytes", c_int64), ("workspace_bytes", c_size_t)]


class muon_bucket_info(ctypes.Structure):
    _fields_ = [("n_matrices", c_int64), ("bytes", c_int64), ("n_groups", c_int64),
                ("m", c_int64), ("n", c_int64), ("ns_single_kernel", c_int64),
                ("momentum_in_ns_kernel", c_int64)]


class muon_bucket_stats(ctypes.Structure):
    _fields_ = [("n_matrices", c_int64), ("n_groups", c_int64), ("m", c_int64), ("n", c_int64),
                ("bytes", c_int64), ("ns_workspace_bytes", c_int64), ("prep_ms", ctypes.c_double),
                ("ns_ms", ctypes.c_double), ("apply_ms", ctypes.c_double), ("h2d_ms", ctypes.c_double),
                ("d2h_ms", ctypes.c_double), ("h2d_bytes", c_int64), ("d2h_bytes", c_int64)]


class muon_stats(ctypes.Structure):
    _fields_ = [("prep_ms", ctypes.c_double), ("ns_ms", ctypes.c_double), ("apply_ms", ctypes.c_double),
                ("h2d_ms", ctypes.c_double), ("d2h_ms", ctypes.c_double), ("step_ms", ctypes.c_double),
                ("h2d_bytes", c_int64), ("d2h_bytes", c_int64), ("n_buckets", c_int64)]


class muon_grad(ctypes.Structure):
    _fields_ = [("g", c_void_p), ("out", c_void_p), ("elems", c_int64), ("count", c_int64),
                ("stride_elems", c_int64), ("dtype", c_int32), ("out_dtype", c_int32)]


class muon_token_batch(ctypes.Structure):
    _fields_ = [("logits", c_void_p), ("targets", c_void_p), ("mask", c_void_p), ("tokens", c_int64),
                ("vocab", c_int64), ("row_stride", c_int64), ("temperature", ctypes.c_double), ("dtype", c_int32),
                ("reserved", c_int32)]


class muon_policy_config(ctypes.Structure):
    _fields_ = [("clip_low", c_float), ("clip_high", c_float), ("kl_beta", c_float), ("grad_scale", c_float),
                ("reduction", c_int32), ("reserved", c_int32 * 3)]


class muon_preference_config(ctypes.Structure):
    _fields_ = [("beta", c_float), ("label_smoothing", c_float), ("grad_scale", c_float),
                ("length_normalize", c_int32), ("reserved", c_int32 * 4)]


def _load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{os.path.basename(path)} not found at {path}; run __graft_entry__.build() "
                          "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    P = c_void_p
    sig = {
        "muon_config_default": (None, [POINTER(muon_config)]),
        "muon_plan": (c_int32, [POINTER(muon_shape), c_int32, POINTER(c_int32), c_int64,
                                POINTER(muon_config), POINTER(P)]),
        "muon_plan_workspace_bytes": (c_int32, [P, POINTER(c_size_t)]),
        "muon_plan_bind_workspace": (c_int32, [P, P, c_size_t]),
        "muon_step": (c_int32, [P, POINTER(P), POINTER(P), POINTER(P), c_int64, c_float, c_float,
                                c_int32, c_float, c_int32, P]),
        "muon_offload_step": (c_int32, [P, POINTER(P), POINTER(P), POINTER(P), c_int64, c_float,
                                        c_int32, c_int32, P, P, c_int64]),
        "muon_sync": (c_int32, [P, P, POINTER(c_int64)]),
        "muon_selftest_wait_timeout": (c_int32, [P, c_int64, P]),
        "muon_get_plan_info": (c_int32, [P, POINTER(muon_plan_info)]),
        "muon_get_bucket_info": (c_int32, [P, c_int64, POINTER(muon_bucket_info)]),
        "muon_set_ns_schedule": (c_int32, [P, POINTER(c_float), c_int32]),
        "muon_polar_express_coefficients": (c_int32, [c_int32, ctypes.c_double, ctypes.c_double,
                                                      POINTER(c_float), POINTER(ctypes.c_double)]),
        "muon_get_stats": (c_int32, [P, POINTER(muon_stats)]),
        "muon_last_error": (c_char_p, []),
        "muon_status_string": (c_char_p, [c_int32]),
        "muon_plan_destroy": (None, [P]),
        "muon_step_noalloc": (c_int32, [P, POINTER(P), POINTER(P), POINTER(P), c_int64, c_float, c_float,
                                        c_int32, c_float, c_int32, P]),
        "muon_noalloc_scratch_bytes": (c_size_t, []),
        "muon_inject_copy_failure": (c_int32, [P, c_int64]),
        "muon_get_bucket_stats": (c_int32, [P, c_int64, POINTER(muon_bucket_stats)]),
        "muon_get_input_norms": (c_int32, [P, POINTER(c_float), c_int64, P]),
        "muon_clip_workspace_bytes": (c_int32, [P, c_int64, POINTER(c_size_t)]),
        "muon_grad_norm": (c_int32, [P, c_int64, P, P, c_size_t, P]),
        "muon_clip_grad_norm": (c_int32, [P, c_int64, c_float, c_float, c_int32, P, P, c_size_t, P]),
        "muon_token_logprobs": (c_int32, [POINTER(muon_token_batch), P, P]),
        "muon_loss_workspace_bytes": (c_int32, [c_int64, c_int64, POINTER(c_size_t)]),
        "muon_policy_config_default": (None, [POINTER(muon_policy_config)]),
        "muon_policy_loss": (c_int32, [POINTER(muon_token_batch), POINTER(muon_policy_config), P, P, P, P, c_int64,
                                       P, P, P, c_int64, P, c_size_t, P]),
        "muon_preference_config_default": (None, [POINTER(muon_preference_config)]),
        "muon_preference_loss": (c_int32, [POINTER(muon_token_batch), POINTER(muon_preference_config), P, P, c_int64,
                                           P, P, P, P, c_int64, P, c_size_t, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_LIB = None


def _lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        _LIB = _load()
    return _LIB


_LIB_DEBUG = False


def use_debug_library(on: bool = True) -> None:
    """Route every later call to libmuon_debug.so (device range checks that record
    MUON_ERR_DEVICE instead of touching memory out of range) or back to libmuon.so.
    A plan belongs to the library that made it: switch only when no plan is alive."""
    global _LIB, _LIB_DEBUG
    _LIB = _load(LIB_PATH_DEBUG if on else LIB_PATH)
    _LIB_DEBUG = bool(on)


def using_debug_library() -> bool:
    return _LIB is not None and _LIB_DEBUG


def __getattr__(name):
    if name == "lib":
        return _lib()
    raise AttributeError(name)


class MuonError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib().muon_last_error().decode() or _lib().muon_status_string(status).decode()
        super().__init__(f"{where}: {_lib().muon_status_string(status).decode()} ({status}): {msg}")


def _check(status: int, where: str) -> int:
    if status < 0:
        raise MuonError(status, where)
    return status


def muon_config_default(**overrides) -> muon_config:
    """The library's default configuration, with fields overridden by keyword."""
    cfg = muon_config()
    _lib().muon_config_default(byref(cfg))
    for k, v in overrides.items():
        if not hasattr(cfg, k):
            raise AttributeError(f"muon_config has no field {k!r}")
        setattr(cfg, k, v)
    return cfg


class Plan:
    """Owner of a muon_plan_t* (destroyed with the object) and its bound workspace."""

    def __init__(self, handle: int, n_tensors: int):
        self.handle = c_void_p(handle)
        self.n_tensors = n_tensors
        self.workspace = None

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            _lib().muon_plan_destroy(h)
            self.handle = c_void_p(0)


def _stream_ptr(stream) -> c_void_p:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return c_void_p(int(getattr(stream, "cuda_stream", stream)))


def _ptrs(tensors) -> ctypes.Array:
    arr = (c_void_p * len(tensors))()
    for i, t in enumerate(tensors):
        arr[i] = c_void_p(t.data_ptr() if hasattr(t, "data_ptr") else int(t))
    return arr


def muon_plan(shapes: Sequence[Sequence[int]], groups: Optional[Sequence[int]] = None,
              bucket_cap_bytes: int = 512 << 20, config: Optional[muon_config] = None) -> Plan:
    """shapes: (rows, cols[, count[, stride_elems]]) per tensor."""
    n = len(shapes)
    arr = (muon_shape * max(n, 1))()
    for i, s in enumerate(shapes):
        s = tuple(int(v) for v in s) + (1, 0)[len(s) - 2:] if len(s) < 4 else tuple(int(v) for v in s)
        arr[i] = muon_shape(s[0], s[1], s[2], s[3])
    g = None
    if groups is not None:
        g = (c_int32 * n)(*[int(v) for v in groups])
    out = c_void_p()
    _check(_lib().muon_plan(arr, n, g, int(bucket_cap_bytes), byref(config) if config is not None else None,
                         byref(out)), "muon_plan")
    return Plan(out.value, n)


def muon_plan_workspace_bytes(plan: Plan) -> int:
    v = c_size_t()
    _check(_lib().muon_plan_workspace_bytes(plan.handle, byref(v)), "muon_plan_workspace_bytes")
    return v.value


def muon_plan_bind_workspace(plan: Plan, workspace) -> None:
    """workspace: a torch uint8 CUDA tensor of at least muon_plan_workspace_bytes bytes."""
    nbytes = workspace.numel() * workspace.element_size()
    _check(_lib().muon_plan_bind_workspace(plan.handle, c_void_p(workspace.data_ptr()), nbytes),
           "muon_plan_bind_workspace")
    plan.workspace = workspace


def muon_step(plan: Plan, params, grads, momentum, lr: float, mu: float, nesterov: bool, wd: float,
              ns_steps: int = 5, stream=None) -> None:
    n = len(params)
    _check(_lib().muon_step(plan.handle, _ptrs(params), _ptrs(grads), _ptrs(momentum), n, float(lr),
                         float(mu), int(bool(nesterov)), float(wd), int(ns_steps), _stream_ptr(stream)),
           "muon_step")


def muon_step_noalloc(plan: Plan, params, grads, momentum, lr: float, mu: float, nesterov: bool,
                      wd: float, ns_steps: int = 5, stream=None) -> None:
    """muon_step without a caller-bound workspace, for callers that cannot allocate
    device memory: the step runs in the library's static device scratch."""
    n = len(params)
    _check(_lib().muon_step_noalloc(plan.handle, _ptrs(params), _ptrs(grads), _ptrs(momentum), n,
                                    float(lr), float(mu), int(bool(nesterov)), float(wd), int(ns_steps),
                                    _stream_ptr(stream)),
           "muon_step_noalloc")


def muon_inject_copy_failure(plan: Plan, nth: int) -> None:
    """The nth host-link copy of the plan's next offload step reports a failure
    (MUON_ERR_CUDA) instead of being enqueued; -1 clears it."""
    _check(_lib().muon_inject_copy_failure(plan.handle, int(nth)), "muon_inject_copy_failure")


def muon_noalloc_scratch_bytes() -> int:
    return int(_lib().muon_noalloc_scratch_bytes())


def muon_offload_step(plan: Plan, h_grads, h_momentum, h_update_out, mu: float, nesterov: bool,
                      ns_steps: int = 5, compute=None, copy=None, timeout_ms: int = 600_000) -> None:
    n = len(h_grads)
    _check(_lib().muon_offload_step(plan.handle, _ptrs(h_grads), _ptrs(h_momentum), _ptrs(h_update_out), n,
                                 float(mu), int(bool(nesterov)), int(ns_steps), _stream_ptr(compute),
                                 c_void_p(int(getattr(copy, "cuda_stream", copy))) if copy is not None
                                 else c_void_p(0), int(timeout_ms)),
           "muon_offload_step")


def muon_sync(plan: Plan, stream=None):
    """Returns (status, n_nonfinite); raises on errors (a device wait that ran out)."""
    nf = c_int64()
    st = _check(_lib().muon_sync(plan.handle, _stream_ptr(stream), byref(nf)), "muon_sync")
    return st, nf.value


def muon_selftest_wait_timeout(plan: Plan, limit_us: int, stream=None) -> None:
    """Enqueue the failure-path self-test: a one-CTA kernel whose bounded wait runs
    out after limit_us; the next muon_sync reports it (MUON_ERR_DEVICE)."""
    _check(_lib().muon_selftest_wait_timeout(plan.handle, int(limit_us), _stream_ptr(stream)),
           "muon_selftest_wait_timeout")


def muon_get_plan_info(plan: Plan) -> muon_plan_info:
    info = muon_plan_info()
    _check(_lib().muon_get_plan_info(plan.handle, byref(info)), "muon_get_plan_info")
    return info


def muon_get_bucket_info(plan: Plan, b: int) -> muon_bucket_info:
    info = muon_bucket_info()
    _check(_lib().muon_get_bucket_info(plan.handle, int(b), byref(info)), "muon_get_bucket_info")
    return info


def muon_set_ns_schedule(plan: Plan, coeffs) -> None:
    """Per-iteration (a, b, c) triples for later steps of the plan; [] restores the
    configuration's coefficients for every iteration."""
    flat = [float(v) for t in coeffs for v in t]
    n = len(flat) // 3
    if n * 3 != len(flat):
        raise ValueError("coefficients are (a, b, c) triples")
    arr = (c_float * max(len(flat), 1))(*flat)
    _check(_lib().muon_set_ns_schedule(plan.handle, arr if n else None, n), "muon_set_ns_schedule")


def muon_polar_express_coefficients(n_iters: int, lower: float = 1e-3, safety: float = 1.0):
    """(coefficient triples, per-iteration error bounds) of the minimax schedule,
    computed by the library on the host."""
    out = (c_float * (3 * int(n_iters)))()
    err = (ctypes.c_double * int(n_iters))()
    _check(_lib().muon_polar_express_coefficients(int(n_iters), float(lower), float(safety), out, err),
           "muon_polar_express_coefficients")
    return [tuple(out[3 * k:3 * k + 3]) for k in range(int(n_iters))], list(err)


def muon_get_stats(plan: Plan) -> muon_stats:
    st = muon_stats()
    _check(_lib().muon_get_stats(plan.handle, byref(st)), "muon_get_stats")
    return st


def muon_get_bucket_stats(plan: Plan, b: int) -> muon_bucket_stats:
    st = muon_bucket_stats()
    _check(_lib().muon_get_bucket_stats(plan.handle, int(b), byref(st)), "muon_get_bucket_stats")
    return st


def muon_get_input_norms(plan: Plan, stream=None):
    """||V||_F of every matrix's Newton-Schulz input in the last step, tensor order."""
    n = int(muon_get_plan_info(plan).n_matrices)
    out = (c_float * n)()
    _check(_lib().muon_get_input_norms(plan.handle, out, n, _stream_ptr(stream)), "muon_get_input_norms")
    return list(out)


def muon_status_string(status: int) -> str:
    return _lib().muon_status_string(int(status)).decode()


def allocate_workspace(plan: Plan, device=None):
    """torch-allocated workspace (256-byte aligned), bound to the plan."""
    import torch
    nbytes = muon_plan_workspace_bytes(plan)
    ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device or "cuda")
    muon_plan_bind_workspace(plan, ws)
    return ws


# ---------------------------------------------------------------------------
# losses on token log-probabilities, and clipping by the global gradient norm
# ---------------------------------------------------------------------------
_NO_CONTEXT = contextlib.nullcontext()


def _on_stream(stream, device: int):
    """(context of a call on `stream`, cudaStream_t).  In the context the tensors' device is the
    current one, on which the library launches, and the allocator hands the memory of the
    tensors that the call allocates out again in the order of the stream that uses it."""
    import torch
    if stream is None:
        context = _NO_CONTEXT if device == torch.cuda.current_device() else torch.cuda.device(device)
        # current_stream(device).cuda_stream without the Stream object
        return context, torch._C._cuda_getCurrentRawStream(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)
    elif stream.device.index != device:
        raise ValueError(f"stream: expected one of cuda:{device}, got one of {stream.device}")
    return torch.cuda.stream(stream), stream.cuda_stream


_DTYPE_CODES: dict = {}


def _dtype_code(dtype) -> int:
    if not _DTYPE_CODES:
        import torch
        _DTYPE_CODES.update({torch.float32: MUON_DTYPE_F32, torch.bfloat16: MUON_DTYPE_BF16})
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        raise TypeError(f"expected a float32 or bfloat16 tensor, got {dtype}")
    return code


def _blocks(t):
    """(elements, count, stride) of a tensor whose memory is `count` equal blocks a stride
    apart, each dense in some order of its dimensions; ValueError otherwise."""
    if t.is_contiguous():
        return t.numel(), 1, 0
    if t.numel() == 0:
        return 0, 0, 0
    elems, outer = 1, None
    for stride, size in sorted(d for d in zip(t.stride(), t.shape) if d[1] != 1):
        if outer is None and stride == elems:
            elems *= size
        elif outer is None and stride > elems:
            outer = (size, stride)
        elif outer is not None and stride == outer[0] * outer[1]:
            outer = (outer[0] * size, outer[1])
        else:
            raise ValueError(f"gradient of shape {tuple(t.shape)} and strides {t.stride()} is not equal dense blocks "
                             "a stride apart")
    return (elems, 1, 0) if outer is None else (elems, outer[0], outer[1])


def _same_layout(g, o):
    """Whether o's elements lie as g's do: its shape and strides (where they matter), or both
    contiguous with as many elements."""
    if g.is_contiguous() and o.is_contiguous():
        return g.numel() == o.numel()
    return g.shape == o.shape and all(a == b or n == 1 for a, b, n in zip(g.stride(), o.stride(), g.shape))


class GradSet:
    """Gradient tensors (and where their clipped values go) as the library takes them.  A
    program whose gradients stay in place makes one and passes it to every call.  An output
    has its gradient's shape and strides, or as many elements where both are contiguous."""

    def __init__(self, grads, out=None):
        import torch
        grads = list(grads)
        out = grads if out is None else list(out)
        n = len(grads)
        if len(out) != n:
            raise ValueError(f"{n} gradients, but {len(out)} outputs")
        self.tensors, self.out = grads, out
        # muon_grad entries, filled field by field (six 8-byte words each): a set may have
        # thousands of tensors
        words = array.array("q", bytes(ctypes.sizeof(muon_grad) * max(n, 1)))
        tensor = torch.Tensor
        codes, devices, dense = _describe(grads)
        words[0::6] = _words(map(tensor.data_ptr, grads), n)
        if dense:
            words[2::6] = _words(map(tensor.numel, grads), n)
            words[3::6] = _words([1] * n, n)
        else:
            for i, g in enumerate(grads):
                words[6 * i + 2], words[6 * i + 3], words[6 * i + 4] = _blocks(g)
        if out is grads:
            words[1::6] = words[0::6]
            words[5::6] = _words([c | c << 32 for c in codes], n)
        else:
            out_codes, out_devices, out_dense = _describe(out)
            devices |= out_devices
            words[1::6] = _words(map(tensor.data_ptr, out), n)
            words[5::6] = _words([c | o << 32 for c, o in zip(codes, out_codes)], n)
            if not dense or not out_dense or words[2::6] != _words(map(tensor.numel, out), n):
                for i, (g, o) in enumerate(zip(grads, out)):
                    if not _same_layout(g, o):
                        raise ValueError(f"gradient {i}: out has another layout")
        if -1 in devices or len(devices) > 1:
            raise ValueError("gradients and outputs must be CUDA tensors of one device")
        self._words = words
        self.array = c_void_p(words.buffer_info()[0])
        self.device = devices.pop() if n else torch.cuda.current_device()

    def __len__(self):
        return len(self.tensors)


def _describe(tensors):
    """(dtype codes, devices (-1: the CPU), whether all are contiguous), with few steps a tensor."""
    import torch
    if not _DTYPE_CODES:
        _dtype_code(torch.float32)
    codes = list(map(_DTYPE_CODES.get, [t.dtype for t in tensors]))
    if None in codes:
        _dtype_code(tensors[codes.index(None)].dtype)  # raises
    return codes, set(map(torch.Tensor.get_device, tensors)), all(map(torch.Tensor.is_contiguous, tensors))


def _words(values, n):
    w = array.array("q", values)
    return w if n else array.array("q", [0])


def muon_clip_workspace_bytes(grads) -> int:
    grads = grads if isinstance(grads, GradSet) else GradSet(grads)
    v = c_size_t()
    _check(_lib().muon_clip_workspace_bytes(grads.array, len(grads), byref(v)), "muon_clip_workspace_bytes")
    return v.value


def _vector(t, n, dtype, what, device):
    """Device pointer of a contiguous tensor of n elements of `dtype` on CUDA device `device`."""
    if t.dtype is not dtype or t.numel() != n or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor of {n} {dtype} values on cuda:{device}, got shape "
                         f"{tuple(t.shape)}, strides {t.stride()}, {t.dtype} on {t.device}")
    return t.data_ptr()


_SPACES = threading.local()  # .held: {(device, stream): workspace}


def _space(workspace, nbytes, device: int, handle: int):
    """(pointer, bytes) of a call's workspace: the caller's, or one that this thread holds for
    the stream, whose calls follow one another.  A call that is being captured, whose graph
    may run beside them, gets one of its own from the capture's memory."""
    import torch
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected a contiguous tensor on cuda:{device}, got {workspace.device}")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if torch.cuda.is_current_stream_capturing():
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), nbytes
    held = _SPACES.__dict__.setdefault("held", {})
    got = held.get((device, handle))
    if got is None or got[2] < nbytes:
        size = max(nbytes, 1 << 17)
        workspace = torch.empty(size, dtype=torch.uint8, device=device)
        got = held[device, handle] = (workspace, workspace.data_ptr(), size)
    return got


def muon_grad_norm(grads, norm=None, workspace=None, stream=None):
    """The global L2 norm of the gradients (a list of tensors or a GradSet), as a
    one-element fp32 device tensor."""
    import torch
    grads = grads if isinstance(grads, GradSet) else GradSet(grads)
    device = grads.device
    nbytes = muon_clip_workspace_bytes(grads)
    context, handle = _on_stream(stream, device)
    with context:
        _keep, ws, nbytes = _space(workspace, nbytes, device, handle)
        if norm is None:
            norm = torch.empty(1, dtype=torch.float32, device=device)
        _check(_lib().muon_grad_norm(grads.array, len(grads), _vector(norm, 1, torch.float32, "norm", device), ws,
                                     nbytes, handle), "muon_grad_norm")
    return norm


def muon_clip_grad_norm(grads, max_norm: float, out=None, eps: float = 1e-6,
                        nonfinite: int = MUON_NONFINITE_KEEP, result=None, workspace=None, stream=None):
    """Scales the gradients (a list of tensors or a GradSet) by min(1, max_norm / (norm + eps)),
    in place or into `out` (a list of tensors of the same layouts, bf16 or fp32).  Returns
    a two-element fp32 device tensor: the norm and the factor."""
    import torch
    if not isinstance(grads, GradSet):
        grads = GradSet(grads, out)
    elif out is not None:
        raise ValueError("a GradSet has its outputs already")
    device = grads.device
    nbytes = muon_clip_workspace_bytes(grads)
    context, handle = _on_stream(stream, device)
    with context:
        _keep, ws, nbytes = _space(workspace, nbytes, device, handle)
        if result is None:
            result = torch.empty(2, dtype=torch.float32, device=device)
        _check(_lib().muon_clip_grad_norm(grads.array, len(grads), max_norm, eps, nonfinite,
                                          _vector(result, 2, torch.float32, "result", device), ws, nbytes, handle),
               "muon_clip_grad_norm")
    return result


def _rows(t, what):
    """(rows, columns, row stride) of a matrix whose rows are contiguous and do not overlap."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{what}: expected a CUDA matrix [tokens, vocab], got shape {tuple(t.shape)} on {t.device}")
    tokens, vocab = t.shape
    stride, inner = t.stride()
    if (vocab > 1 and inner != 1) or (tokens > 1 and stride < vocab):
        raise ValueError(f"{what}: rows must be contiguous and not overlap, got strides {t.stride()}")
    return tokens, vocab, stride if tokens > 1 else vocab


def _token_batch(logits, targets, mask, temperature):
    """(muon_token_batch, tokens, vocab, row stride, device)"""
    import torch
    tokens, vocab, stride = _rows(logits, "logits")
    device = logits.get_device()
    masked = None
    if mask is not None:
        if mask.dtype is not torch.bool and mask.dtype is not torch.uint8:
            raise ValueError(f"mask: expected bool or uint8, got {mask.dtype}")
        masked = _vector(mask, tokens, mask.dtype, "mask", device)
    return muon_token_batch(logits.data_ptr(), _vector(targets, tokens, torch.int64, "targets", device), masked, tokens,
                            vocab, stride, temperature, _dtype_code(logits.dtype)), tokens, vocab, stride, device


def _grad_rows(logits, grad, with_grad, tokens, vocab, stride):
    """(gradient tensor or None, its pointer, its row stride): by default with the logits'
    row stride, so that both start on the same boundaries, unless that would waste memory."""
    import torch
    if grad is None:
        if not with_grad:
            return None, None, 0
        if stride > vocab + vocab // 8:
            stride = vocab
        grad = torch.empty_strided((tokens, vocab), (stride, 1), dtype=logits.dtype, device=logits.device)
        return grad, grad.data_ptr(), stride
    if grad.shape != logits.shape or grad.dtype is not logits.dtype or grad.get_device() != logits.get_device():
        raise ValueError(f"grad: expected a tensor like the logits, got shape {tuple(grad.shape)}, {grad.dtype} "
                         f"on {grad.device}")
    return grad, grad.data_ptr(), _rows(grad, "grad")[2]


def muon_token_logprobs(logits, targets, mask=None, temperature: float = 1.0, logp=None, stream=None):
    """log softmax(logits / temperature) at each position's target, fp32; 0 where the mask
    is False.  logits: [tokens, vocab], targets: [tokens] int64, mask: [tokens] bool."""
    import torch
    batch, tokens, _, _, device = _token_batch(logits, targets, mask, temperature)
    context, handle = _on_stream(stream, device)
    with context:
        if logp is None:
            logp = torch.empty(tokens, dtype=torch.float32, device=device)
        _check(_lib().muon_token_logprobs(byref(batch), _vector(logp, tokens, torch.float32, "logp", device), handle),
               "muon_token_logprobs")
    return logp


def muon_loss_workspace_bytes(tokens: int, n_seqs: int) -> int:
    v = c_size_t()
    _check(_lib().muon_loss_workspace_bytes(int(tokens), int(n_seqs), byref(v)), "muon_loss_workspace_bytes")
    return v.value


def _default_config(cls, default, overrides):
    cfg = cls()
    default(byref(cfg))
    for k, v in overrides.items():
        if not hasattr(cfg, k):
            raise AttributeError(f"{cls.__name__} has no field {k!r}")
        setattr(cfg, k, v)
    return cfg


def muon_policy_config_default(**overrides) -> muon_policy_config:
    return _default_config(muon_policy_config, _lib().muon_policy_config_default, overrides)


def muon_preference_config_default(**overrides) -> muon_preference_config:
    return _default_config(muon_preference_config, _lib().muon_preference_config_default, overrides)


def muon_policy_loss(logits, targets, old_logp, advantages, mask=None, ref_logp=None, seq_offsets=None,
                     temperature: float = 1.0, config: Optional[muon_policy_config] = None, grad=None, logp=None,
                     stats=None, with_grad: bool = True, workspace=None, stream=None):
    """The clipped policy loss with a KL term, and its gradient with respect to the logits.

    Returns (stats, logp, grad): stats holds the loss, the policy term, the KL term and the
    clipped share (fp32, on the device); grad is None with with_grad=False.  seq_offsets:
    [n_seqs + 1] int64, for the sequence mean.  grad may be the logits themselves."""
    import torch
    f32 = torch.float32
    batch, tokens, vocab, stride, device = _token_batch(logits, targets, mask, temperature)
    n_seqs, offsets = 0, None
    if seq_offsets is not None:
        n_seqs = max(seq_offsets.numel() - 1, 0)
        offsets = _vector(seq_offsets, n_seqs + 1, torch.int64, "seq_offsets", device)
    context, handle = _on_stream(stream, device)
    with context:
        _keep, ws, nbytes = _space(workspace, muon_loss_workspace_bytes(tokens, n_seqs), device, handle)
        if stats is None:
            stats = torch.empty(4, dtype=f32, device=device)
        if logp is None:
            logp = torch.empty(tokens, dtype=f32, device=device)
        grad, grad_ptr, grad_stride = _grad_rows(logits, grad, with_grad, tokens, vocab, stride)
        _check(_lib().muon_policy_loss(
            byref(batch), byref(config) if config is not None else None,
            _vector(old_logp, tokens, f32, "old_logp", device),
            None if ref_logp is None else _vector(ref_logp, tokens, f32, "ref_logp", device),
            _vector(advantages, tokens, f32, "advantages", device), offsets, n_seqs,
            _vector(stats, 4, f32, "stats", device), _vector(logp, tokens, f32, "logp", device), grad_ptr, grad_stride,
            ws, nbytes, handle), "muon_policy_loss")
    return stats, logp, grad


def muon_preference_loss(logits, targets, seq_offsets, ref_logp, mask=None, temperature: float = 1.0,
                         config: Optional[muon_preference_config] = None, grad=None, loss=None, margins=None,
                         seq_logp=None, with_grad: bool = True, workspace=None, stream=None):
    """The preference loss over pairs of sequences, and its gradient with respect to the logits.

    seq_offsets: [2 P + 1] int64: the P preferred answers, then the P others.  ref_logp:
    [2 P] fp32, the reference policy's sums.  Returns (loss, margins, seq_logp, grad)."""
    import torch
    f32 = torch.float32
    batch, tokens, vocab, stride, device = _token_batch(logits, targets, mask, temperature)
    n_seqs = seq_offsets.numel() - 1
    if n_seqs < 0 or n_seqs % 2:
        raise ValueError(f"seq_offsets: expected 2 P + 1 offsets, got {seq_offsets.numel()}")
    context, handle = _on_stream(stream, device)
    with context:
        _keep, ws, nbytes = _space(workspace, muon_loss_workspace_bytes(tokens, n_seqs), device, handle)
        if loss is None and margins is None and seq_logp is None:  # one allocation for the three
            loss, margins, seq_logp = torch.empty(1 + 3 * (n_seqs // 2), dtype=f32, device=device).split_with_sizes(
                (1, n_seqs // 2, n_seqs))
        if loss is None:
            loss = torch.empty(1, dtype=f32, device=device)
        if margins is None:
            margins = torch.empty(n_seqs // 2, dtype=f32, device=device)
        if seq_logp is None:
            seq_logp = torch.empty(n_seqs, dtype=f32, device=device)
        grad, grad_ptr, grad_stride = _grad_rows(logits, grad, with_grad, tokens, vocab, stride)
        _check(_lib().muon_preference_loss(
            byref(batch), byref(config) if config is not None else None,
            _vector(ref_logp, n_seqs, f32, "ref_logp", device),
            _vector(seq_offsets, n_seqs + 1, torch.int64, "seq_offsets", device), n_seqs // 2,
            _vector(loss, 1, f32, "loss", device), _vector(margins, n_seqs // 2, f32, "margins", device),
            _vector(seq_logp, n_seqs, f32, "seq_logp", device), grad_ptr, grad_stride, ws, nbytes, handle),
            "muon_preference_loss")
    return loss, margins, seq_logp, grad
