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


class muon_checkpoint(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("rows", c_int64), ("cols", c_int64)]


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
        "muon_sample_workspace_bytes": (c_int32, [c_int64, c_int64, c_int32, POINTER(c_size_t)]),
        "muon_sample_tokens": (c_int32, [POINTER(muon_token_batch), P, P, P, P, c_size_t, P]),
        "muon_verify_drafts": (c_int32, [POINTER(muon_token_batch), POINTER(muon_token_batch), P, P, c_int64, P, P,
                                         P, P, P, P, c_size_t, P]),
        "muon_checkpoint_bytes": (c_int32, [c_int64, c_int64, POINTER(c_size_t)]),
        "muon_checkpoint_save": (c_int32, [P, c_int64, c_int32, POINTER(muon_checkpoint), P]),
        "muon_checkpoint_load": (c_int32, [POINTER(muon_checkpoint), P, c_int64, c_int32, P]),
        "muon_weight_grad_workspace_bytes": (c_int32, [POINTER(muon_checkpoint), P, c_int64, c_int32, c_int64,
                                                       POINTER(c_size_t)]),
        "muon_checkpoint_weight_grad": (c_int32, [POINTER(muon_checkpoint), P, c_int64, c_int32, c_int64, P, c_int64,
                                                  c_int32, c_int32, P, c_size_t, P]),
        "muon_swiglu_forward": (c_int32, [P, c_int64, P, c_int64, c_int32, P, c_int64, POINTER(muon_checkpoint),
                                          POINTER(muon_checkpoint), P]),
        "muon_swiglu_backward": (c_int32, [P, c_int64, c_int32, POINTER(muon_checkpoint), POINTER(muon_checkpoint), P,
                                           c_int64, P, c_int64, P, c_int64, P]),
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
_MOST_HELD = 1 << 25         # bytes of one


def _space(workspace, nbytes, device: int, handle: int):
    """(workspace, pointer, bytes) of a call: the caller's, or one that this thread holds for the
    stream, whose calls follow one another.  One of more than _MOST_HELD bytes is the call's
    own: the allocator has it back, in the stream's order, when the call returns.  A call that is
    being captured, whose graph may run beside the others, gets one from the capture's memory."""
    import torch
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected a contiguous tensor on cuda:{device}, got {workspace.device}")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if nbytes > _MOST_HELD or torch.cuda.is_current_stream_capturing():
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


def _mask_type(mask):
    import torch
    if mask.dtype is not torch.bool and mask.dtype is not torch.uint8:
        raise ValueError(f"mask: expected bool or uint8, got {mask.dtype}")
    return mask.dtype


def _token_batch(logits, targets, mask, temperature):
    """(muon_token_batch, tokens, vocab, row stride, device)"""
    import torch
    tokens, vocab, stride = _rows(logits, "logits")
    device = logits.get_device()
    masked = None
    if mask is not None:
        masked = _vector(mask, tokens, _mask_type(mask), "mask", device)
    return muon_token_batch(logits.data_ptr(), _vector(targets, tokens, torch.int64, "targets", device), masked, tokens,
                            vocab, stride, temperature, _dtype_code(logits.dtype)), tokens, vocab, stride, device


def _row_batch(logits, mask, temperature, what="logits"):
    """(muon_token_batch without targets, rows, device)"""
    rows, vocab, stride = _rows(logits, what)
    device = logits.get_device()
    masked = None
    if mask is not None:
        masked = _vector(mask, rows, _mask_type(mask), "mask", device)
    return muon_token_batch(logits.data_ptr(), None, masked, rows, vocab, stride, temperature,
                            _dtype_code(logits.dtype)), rows, device


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


def muon_sample_workspace_bytes(rows: int, vocab: int, dtype) -> int:
    v = c_size_t()
    _check(_lib().muon_sample_workspace_bytes(rows, vocab, _dtype_code(dtype), byref(v)),
           "muon_sample_workspace_bytes")
    return v.value


def muon_sample_tokens(logits, uniforms, mask=None, temperature: float = 1.0, tokens=None, logp=None, workspace=None,
                       stream=None):
    """A token for each row of logits [rows, vocab], drawn from softmax(logits / temperature)
    with a given uniform number: the first whose cumulated probability exceeds it.  uniforms:
    [rows] fp32 in [0, 1), mask: [rows] bool.  Returns (tokens int64, their log-probabilities
    fp32); -1 and 0 where the mask is False, -1 and NaN in a row without probabilities."""
    import torch
    batch, rows, device = _row_batch(logits, mask, temperature)
    nbytes = muon_sample_workspace_bytes(rows, batch.vocab, logits.dtype)
    context, handle = _on_stream(stream, device)
    with context:
        _keep, ws, nbytes = _space(workspace, nbytes, device, handle)
        if tokens is None:
            tokens = torch.empty(rows, dtype=torch.int64, device=device)
        if logp is None:
            logp = torch.empty(rows, dtype=torch.float32, device=device)
        _check(_lib().muon_sample_tokens(byref(batch), _vector(uniforms, rows, torch.float32, "uniforms", device),
                                         _vector(tokens, rows, torch.int64, "tokens", device),
                                         _vector(logp, rows, torch.float32, "logp", device), ws, nbytes, handle),
               "muon_sample_tokens")
    return tokens, logp


def muon_verify_drafts(logits, drafts, draft_offsets, accept_uniforms, sample_uniforms, draft_logits=None,
                       draft_logp=None, temperature: float = 1.0, draft_temperature: Optional[float] = None,
                       tokens=None, counts=None, logp=None, workspace=None, stream=None):
    """Verifies the drafted tokens of several sequences against the target's probabilities.

    logits: [N + S, vocab], for each sequence a row for each of its drafts and one after them;
    drafts: [N] int64; draft_offsets: [S + 1] int64, ascending from 0 to N; accept_uniforms
    [N] and sample_uniforms [S]: fp32 in [0, 1).  draft_logits: [N, vocab], what the drafts
    were sampled from (None: they were certain), and draft_logp: [N] fp32, their
    log-probabilities under it where they are known.  draft_temperature: by default the
    target's.  Returns (tokens [N + S]: taken drafts, one drawn token, then -1; counts [S] of
    the drafts taken; logp [N + S] of the tokens under the target)."""
    import torch
    f32, i64 = torch.float32, torch.int64
    target, rows, device = _row_batch(logits, None, temperature)
    n_seqs = draft_offsets.numel() - 1
    if n_seqs < 0:
        raise ValueError("draft_offsets: expected S + 1 offsets, got none")
    n = rows - n_seqs
    if draft_temperature is None:
        draft_temperature = temperature
    if draft_logits is None:
        draft = muon_token_batch(None, None, None, n, target.vocab, 0, draft_temperature, target.dtype)
    else:
        draft, got, draft_device = _row_batch(draft_logits, None, draft_temperature, "draft_logits")
        if got != n or draft.vocab != target.vocab or draft.dtype != target.dtype or draft_device != device:
            raise ValueError(f"draft_logits: expected [{n}, {target.vocab}] {logits.dtype} values on cuda:{device}, got "
                             f"shape {tuple(draft_logits.shape)}, {draft_logits.dtype} on {draft_logits.device}")
    draft.targets = _vector(drafts, n, i64, "drafts", device)
    nbytes = muon_sample_workspace_bytes(rows + (0 if draft_logits is None else n), target.vocab, logits.dtype)
    context, handle = _on_stream(stream, device)
    with context:
        _keep, ws, nbytes = _space(workspace, nbytes, device, handle)
        if tokens is None:
            tokens = torch.empty(rows, dtype=i64, device=device)
        if counts is None:
            counts = torch.empty(n_seqs, dtype=i64, device=device)
        if logp is None:
            logp = torch.empty(rows, dtype=f32, device=device)
        _check(_lib().muon_verify_drafts(
            byref(target), byref(draft), None if draft_logp is None else _vector(draft_logp, n, f32, "draft_logp", device),
            _vector(draft_offsets, n_seqs + 1, i64, "draft_offsets", device), n_seqs,
            _vector(accept_uniforms, n, f32, "accept_uniforms", device),
            _vector(sample_uniforms, n_seqs, f32, "sample_uniforms", device), _vector(tokens, rows, i64, "tokens", device),
            _vector(counts, n_seqs, i64, "counts", device), _vector(logp, rows, f32, "logp", device), ws, nbytes,
            handle), "muon_verify_drafts")
    return tokens, counts, logp


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


# ---------------------------------------------------------------------------
# activation checkpoints in 8 bits
# ---------------------------------------------------------------------------
def muon_checkpoint_bytes(rows: int, cols: int) -> int:
    v = c_size_t()
    _check(_lib().muon_checkpoint_bytes(int(rows), int(cols), byref(v)), "muon_checkpoint_bytes")
    return v.value


class Checkpoint:
    """An activation matrix [rows, cols] in 8 bits (include/muon.h, muon_checkpoint).  data: a
    contiguous CUDA uint8 tensor of muon_checkpoint_bytes bytes that starts on a 16-byte
    boundary; by default a new one on `device` (the current one)."""

    def __init__(self, rows: int, cols: int, data=None, device=None):
        import torch
        nbytes = muon_checkpoint_bytes(rows, cols)
        if data is None:
            data = torch.empty(nbytes, dtype=torch.uint8, device="cuda" if device is None else device)
        if data.dtype is not torch.uint8 or data.numel() != nbytes or not data.is_cuda or not data.is_contiguous():
            raise ValueError(f"data: expected a contiguous CUDA tensor of {nbytes} uint8 values, got shape "
                             f"{tuple(data.shape)}, strides {data.stride()}, {data.dtype} on {data.device}")
        self.rows, self.cols, self.data, self.device = rows, cols, data, data.get_device()
        self.struct = muon_checkpoint(data.data_ptr(), rows, cols)

    @property
    def shape(self):
        return self.rows, self.cols


def _saved(checkpoint, rows, cols, device, what="checkpoint"):
    """A given checkpoint of this shape and device, or a new one."""
    if checkpoint is None:
        return Checkpoint(rows, cols, device=device)
    if checkpoint.shape != (rows, cols) or checkpoint.device != device:
        raise ValueError(f"{what}: expected one of [{rows}, {cols}] on cuda:{device}, got one of "
                         f"{list(checkpoint.shape)} on cuda:{checkpoint.device}")
    return checkpoint


def _matrix(t, rows, cols, dtype, device, what):
    """(pointer, row stride) of a matrix whose rows are contiguous and do not overlap."""
    if t.dtype is not dtype or t.shape != (rows, cols) or t.get_device() != device:
        raise ValueError(f"{what}: expected [{rows}, {cols}] {dtype} values on cuda:{device}, got shape {tuple(t.shape)}, "
                         f"{t.dtype} on {t.device}")
    stride, inner = t.stride()
    if (cols > 1 and inner != 1) or (rows > 1 and stride < cols):
        raise ValueError(f"{what}: rows must be contiguous and not overlap, got strides {t.stride()}")
    return t.data_ptr(), stride if rows > 1 else cols


def muon_checkpoint_save(x, checkpoint=None, stream=None):
    """Keeps x [rows, cols] (bf16 or fp32) in 8 bits: int8 values and one power of two for each
    block of 32 columns of a row.  Returns the Checkpoint."""
    rows, cols, stride = _rows(x, "x")
    device, dtype = x.get_device(), _dtype_code(x.dtype)
    context, handle = _on_stream(stream, device)
    with context:
        checkpoint = _saved(checkpoint, rows, cols, device)
        _check(_lib().muon_checkpoint_save(x.data_ptr(), stride, dtype, byref(checkpoint.struct), handle),
               "muon_checkpoint_save")
    return checkpoint


def muon_checkpoint_load(checkpoint, out=None, dtype=None, stream=None):
    """The values of a checkpoint, in `out` or a new matrix of `dtype` (bf16 by default, which
    holds them exactly)."""
    import torch
    rows, cols = checkpoint.shape
    device = checkpoint.device
    context, handle = _on_stream(stream, device)
    with context:
        if out is None:
            out = torch.empty(rows, cols, dtype=dtype or torch.bfloat16, device=device)
        elif dtype is not None and out.dtype is not dtype:
            raise ValueError(f"out: expected {dtype}, got {out.dtype}")
        code = _dtype_code(out.dtype)
        _check(_lib().muon_checkpoint_load(byref(checkpoint.struct), *_matrix(out, rows, cols, out.dtype, device, "out"),
                                           code, handle), "muon_checkpoint_load")
    return out


def muon_weight_grad_workspace_bytes(checkpoint, dy) -> int:
    outs, stride = _gradient_rows(checkpoint, dy)
    v = c_size_t()
    _check(_lib().muon_weight_grad_workspace_bytes(byref(checkpoint.struct), dy.data_ptr(), stride, _dtype_code(dy.dtype),
                                                   outs, byref(v)), "muon_weight_grad_workspace_bytes")
    return v.value


def _gradient_rows(checkpoint, dy):
    """(outs, row stride) of the gradient of a linear layer's output."""
    rows, outs, stride = _rows(dy, "dy")
    if rows != checkpoint.rows or dy.get_device() != checkpoint.device:
        raise ValueError(f"dy: expected {checkpoint.rows} rows on cuda:{checkpoint.device}, got shape {tuple(dy.shape)} on "
                         f"{dy.device}")
    return outs, stride


def muon_checkpoint_weight_grad(checkpoint, dy, out=None, accumulate: bool = False, dtype=None, workspace=None,
                                stream=None):
    """The weight gradient dy^T x [outs, cols] of y = x W^T from the checkpoint of x [rows, cols]
    and dy [rows, outs] (bf16 or fp32), written to `out` or a new matrix of `dtype` (dy's by
    default), or added to `out` with accumulate=True.  Its workspace (muon_weight_grad_workspace_bytes)
    holds x in bf16 and, for fp32 dy, three bf16 copies of dy."""
    import torch
    outs, stride = _gradient_rows(checkpoint, dy)
    cols, device = checkpoint.cols, checkpoint.device
    if out is None and accumulate:
        raise ValueError("accumulate=True needs out")
    if out is not None and dtype is not None and out.dtype is not dtype:
        raise ValueError(f"out: expected {dtype}, got {out.dtype}")
    nbytes = muon_weight_grad_workspace_bytes(checkpoint, dy)
    context, handle = _on_stream(stream, device)
    with context:
        _keep, ws, nbytes = _space(workspace, nbytes, device, handle) if nbytes else (None, None, 0)
        if out is None:
            out = torch.empty(outs, cols, dtype=dtype or dy.dtype, device=device)
        ptr, out_stride = _matrix(out, outs, cols, out.dtype, device, "out")
        _check(_lib().muon_checkpoint_weight_grad(byref(checkpoint.struct), dy.data_ptr(), stride, _dtype_code(dy.dtype),
                                                  outs, ptr, out_stride, _dtype_code(out.dtype), int(bool(accumulate)),
                                                  ws, nbytes, handle), "muon_checkpoint_weight_grad")
    return out


def muon_swiglu_forward(gate, up, h=None, gate_checkpoint=None, up_checkpoint=None, stream=None):
    """h = gate sigmoid(gate) up, and the 8-bit checkpoints of gate and up [rows, cols] (which
    may be halves of one matrix).  Returns (h, gate's Checkpoint, up's Checkpoint)."""
    import torch
    rows, cols, stride = _rows(gate, "gate")
    device, dtype = gate.get_device(), gate.dtype
    code = _dtype_code(dtype)
    context, handle = _on_stream(stream, device)
    with context:
        if h is None:
            h = torch.empty(rows, cols, dtype=dtype, device=device)
        gate_checkpoint = _saved(gate_checkpoint, rows, cols, device, "gate_checkpoint")
        up_checkpoint = _saved(up_checkpoint, rows, cols, device, "up_checkpoint")
        _check(_lib().muon_swiglu_forward(gate.data_ptr(), stride, *_matrix(up, rows, cols, dtype, device, "up"), code,
                                          *_matrix(h, rows, cols, dtype, device, "h"), byref(gate_checkpoint.struct),
                                          byref(up_checkpoint.struct), handle), "muon_swiglu_forward")
    return h, gate_checkpoint, up_checkpoint


def muon_swiglu_backward(dh, gate_checkpoint, up_checkpoint, dgate=None, dup=None, h=None, with_h: bool = False,
                         stream=None):
    """The gradients of muon_swiglu_forward's inputs from h's [rows, cols] and the
    checkpoints.  Returns (dgate, dup, h): h is computed again with with_h=True (or a given
    h), else None.  One of the outputs may be dh itself."""
    import torch
    rows, cols, stride = _rows(dh, "dh")
    device, dtype = dh.get_device(), dh.dtype
    code = _dtype_code(dtype)
    _saved(gate_checkpoint, rows, cols, device, "gate_checkpoint")
    _saved(up_checkpoint, rows, cols, device, "up_checkpoint")
    context, handle = _on_stream(stream, device)
    with context:
        if dgate is None:
            dgate = torch.empty(rows, cols, dtype=dtype, device=device)
        if dup is None:
            dup = torch.empty(rows, cols, dtype=dtype, device=device)
        if h is None and with_h:
            h = torch.empty(rows, cols, dtype=dtype, device=device)
        _check(_lib().muon_swiglu_backward(
            dh.data_ptr(), stride, code, byref(gate_checkpoint.struct), byref(up_checkpoint.struct),
            *_matrix(dgate, rows, cols, dtype, device, "dgate"), *_matrix(dup, rows, cols, dtype, device, "dup"),
            *((None, 0) if h is None else _matrix(h, rows, cols, dtype, device, "h")), handle), "muon_swiglu_backward")
    return dgate, dup, h
