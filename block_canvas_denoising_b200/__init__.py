"""B200 (sm_100a) denoising step of block discrete-diffusion text generation.

A thin ctypes binding of ``libdg.so`` (C ABI in ``include/dg.h``): argument
marshalling only.  Every step of the path runs in the library's CUDA
kernels; PyTorch supplies device memory and streams.  There is no CPU
fallback: if the library is missing or no sm_100 device is present, calls
raise ``DGError``.
"""
from __future__ import annotations

import contextlib
import ctypes
import itertools
import os
from dataclasses import dataclass

import numpy as np

__all__ = ["DGError", "Params", "lib", "workspace_size", "Workspace", "denoise_step",
           "debug_logits", "device_status", "denoise_loop", "debug_gumbel",
           "selftest_bounded_wait", "set_head_events", "denoise_step_noalloc", "noalloc_status",
           "noalloc_selftest_bounded_wait", "STATUS", "E_BF16", "E_FP8_E4M3",
           "SELECT_CUMSUM", "SELECT_MI", "SELECT_TOPK", "partials_count", "head_partials", "merge_partials",
           "gather_partials", "init_canvas", "generate_blocks", "loop_state_bytes", "LoopState",
           "denoise_loop_graph", "selfcond_workspace_size", "embedder_transpose", "denoise_step_selfcond", "PAGE",
           "ContextPlan", "context_plan", "context_status", "RopeFrequencies", "rope", "ContextCache",
           "context_append", "context_workspace_size", "ContextWorkspace", "context_attention",
           "generate_blocks_context"]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg.so")

E_BF16 = 0
E_FP8_E4M3 = 1

STATUS = {0: "DG_OK", 1: "DG_ERR_INVALID_ARG", 2: "DG_ERR_UNSUPPORTED_SHAPE", 3: "DG_ERR_WORKSPACE",
          4: "DG_ERR_RANGE", 5: "DG_ERR_CUDA", 6: "DG_ERR_TIMEOUT", 7: "DG_ERR_CALLBACK",
          8: "DG_ERR_NO_DEVICE", 9: "DG_ERR_VALUE", 10: "DG_ERR_CAPACITY"}


class DGError(RuntimeError):
    def __init__(self, code: int, where: str = ""):
        self.code = int(code)
        super().__init__(f"{where}: {STATUS.get(self.code, self.code)}")


class _Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("L", ctypes.c_int32), ("d", ctypes.c_int32),
                ("V", ctypes.c_int32), ("e_dtype", ctypes.c_int32)]


class _Params(ctypes.Structure):
    _fields_ = [("tau0", ctypes.c_double), ("tau1", ctypes.c_double), ("max_steps", ctypes.c_int32),
                ("entropy_bound", ctypes.c_double), ("stop_entropy", ctypes.c_double),
                ("seed", ctypes.c_uint64), ("selection_rule", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("block", ctypes.c_int32)]


class _Context(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("rows", ctypes.c_int32), ("pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)] + [(n, ctypes.c_void_p) for n in (
                    "table", "held", "free_list", "free_count", "lens", "start", "positions", "slots", "runs",
                    "free_next", "status", "epoch")]


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _RopeArgs(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("freq", ctypes.c_void_p)]


class _Cache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("kept", ctypes.c_void_p)]


SELECT_CUMSUM = 0
SELECT_MI = 1
SELECT_TOPK = 2


_HIDDEN_FN = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                              ctypes.c_void_p, ctypes.c_void_p)
_BLOCK_HIDDEN_FN = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p)


@dataclass
class Params:
    """Sampler parameters (defaults: the serving configuration of the docs)."""
    tau0: float = 0.8
    tau1: float = 0.4
    max_steps: int = 48
    entropy_bound: float = 0.1
    stop_entropy: float = 0.005
    seed: int = 1234
    selection_rule: int = SELECT_CUMSUM
    top_k: int = 1
    block: int = 0

    def c(self) -> _Params:
        return _Params(self.tau0, self.tau1, self.max_steps, self.entropy_bound,
                       self.stop_entropy, int(self.seed) & 0xFFFFFFFFFFFFFFFF,
                       int(self.selection_rule), int(self.top_k), int(self.block))


_lib = None


def lib() -> ctypes.CDLL:
    """Load libdg.so (built in-tree by ``block_canvas_denoising_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise DGError(5, f"libdg.so not built at {LIB_PATH}")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        L.dg_default_params.restype = _Params
        L.dg_error_string.restype = ctypes.c_char_p
        L.dg_error_string.argtypes = [ctypes.c_int]
        L.dg_workspace_size.restype = ctypes.c_size_t
        L.dg_workspace_size.argtypes = [ctypes.POINTER(_Shape)]
        L.dg_workspace_init.argtypes = [P, ctypes.c_size_t, P]
        step_args = [ctypes.POINTER(_Shape), ctypes.POINTER(_Params), P, P, P, P, P, P,
                     P, P, P, P, P, P, P]
        L.dg_denoise_step.argtypes = step_args + [P, ctypes.c_size_t, P]
        L.dg_debug_logits.argtypes = step_args + [P, P, ctypes.c_size_t, P]
        L.dg_device_status.argtypes = [P, ctypes.c_size_t, P]
        L.dg_denoise_loop.argtypes = [ctypes.POINTER(_Shape), ctypes.POINTER(_Params), P, P,
                                      _HIDDEN_FN, P, ctypes.c_int32, P, P, P, P, P,
                                      P, P, P, P, P, P, ctypes.c_size_t, P]
        L.dg_selftest_bounded_wait.argtypes = [ctypes.c_uint64, P, ctypes.c_size_t, P]
        L.dg_debug_gumbel.argtypes = [P, ctypes.c_int32, P, P, P]
        L.dg_set_head_events.argtypes = [P, P]
        L.dg_denoise_step_noalloc.argtypes = step_args + [P]
        L.dg_denoise_step_noalloc.restype = ctypes.c_int
        L.dg_noalloc_status.argtypes = [P]
        L.dg_noalloc_status.restype = ctypes.c_int
        L.dg_noalloc_selftest_bounded_wait.argtypes = [ctypes.c_uint64, P]
        L.dg_noalloc_selftest_bounded_wait.restype = ctypes.c_int
        L.dg_last_error_message.restype = ctypes.c_char_p
        L.dg_selfcond_workspace_size.argtypes = [ctypes.POINTER(_Shape)]
        L.dg_selfcond_workspace_size.restype = ctypes.c_size_t
        L.dg_embedder_transpose.argtypes = [ctypes.POINTER(_Shape), P, P, P]
        L.dg_embedder_transpose.restype = ctypes.c_int
        L.dg_denoise_step_selfcond.argtypes = [ctypes.POINTER(_Shape), ctypes.POINTER(_Params), P, P, P, P, P, P,
                                               P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.dg_denoise_step_selfcond.restype = ctypes.c_int
        L.dg_loop_state_bytes.argtypes = [ctypes.c_int32]
        L.dg_loop_state_bytes.restype = ctypes.c_size_t
        L.dg_denoise_loop_graph.argtypes = [ctypes.POINTER(_Shape), ctypes.POINTER(_Params), P, P, P,
                                            ctypes.c_int32, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P,
                                            ctypes.c_size_t, P]
        L.dg_denoise_loop_graph.restype = ctypes.c_int
        L.dg_loop_graph_create.argtypes = [ctypes.POINTER(_Shape), ctypes.POINTER(_Params), P, P, P, P, P, P,
                                           P, P, P, P, P, P, ctypes.c_size_t, P, ctypes.c_size_t,
                                           ctypes.POINTER(ctypes.c_void_p)]
        L.dg_loop_graph_create.restype = ctypes.c_int
        L.dg_loop_graph_run.argtypes = [P, ctypes.c_int32, P, P, P]
        L.dg_loop_graph_run.restype = ctypes.c_int
        L.dg_loop_graph_destroy.argtypes = [P]
        L.dg_loop_graph_destroy.restype = None
        L.dg_init_canvas.argtypes = [ctypes.POINTER(_Shape), ctypes.POINTER(_Params), P, P]
        L.dg_init_canvas.restype = ctypes.c_int
        L.dg_generate_blocks.argtypes = [ctypes.POINTER(_Shape), ctypes.POINTER(_Params), P, P, ctypes.c_int32,
                                         _BLOCK_HIDDEN_FN, P, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.dg_generate_blocks.restype = ctypes.c_int
        gb = list(L.dg_generate_blocks.argtypes)
        L.dg_generate_blocks_context.argtypes = gb[:7] + [P, P] + gb[7:]
        L.dg_generate_blocks_context.restype = ctypes.c_int
        L.dg_context_plan.argtypes = [P, P, P, ctypes.c_int32, P]
        L.dg_context_plan.restype = ctypes.c_int
        L.dg_context_status.argtypes = [P, P]
        L.dg_context_status.restype = ctypes.c_int
        L.dg_rope_frequencies.argtypes = [ctypes.c_int32, ctypes.c_double, ctypes.c_int32, ctypes.c_double,
                                          ctypes.c_int32, P, P]
        L.dg_rope_frequencies.restype = ctypes.c_int
        L.dg_rope.argtypes = [P, P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, P, P]
        L.dg_rope.restype = ctypes.c_int
        L.dg_context_kept_size.argtypes = [ctypes.c_int32] * 3
        L.dg_context_kept_size.restype = ctypes.c_size_t
        L.dg_context_append.argtypes = [P, P, P, P, P, P]
        L.dg_context_append.restype = ctypes.c_int
        L.dg_context_workspace_size.argtypes = [ctypes.c_int32] * 4
        L.dg_context_workspace_size.restype = ctypes.c_size_t
        L.dg_context_attention.argtypes = [P, P, P, P, ctypes.c_int32, ctypes.c_float, P, ctypes.c_int32,
                                           ctypes.c_int32, P, P, ctypes.c_size_t, P]
        L.dg_context_attention.restype = ctypes.c_int
        L.dg_partials_count.restype = ctypes.c_int32
        L.dg_partials_count.argtypes = [ctypes.POINTER(_Shape)]
        L.dg_head_partials.restype = ctypes.c_int
        L.dg_head_partials.argtypes = [ctypes.POINTER(_Shape), ctypes.POINTER(_Params), ctypes.c_int32,
                                       P, P, P, P, P, P, ctypes.c_size_t, P]
        L.dg_merge_partials.restype = ctypes.c_int
        L.dg_merge_partials.argtypes = [ctypes.POINTER(_Shape), ctypes.POINTER(_Params), P, ctypes.c_int32,
                                        ctypes.c_int32, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        for name in ("dg_workspace_init", "dg_denoise_step", "dg_debug_logits", "dg_device_status",
                     "dg_denoise_loop", "dg_selftest_bounded_wait", "dg_debug_gumbel",
                     "dg_set_head_events"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(code: int, where: str) -> None:
    if code != 0:
        msg = lib().dg_last_error_message().decode(errors="replace")
        raise DGError(code, where + (f" [{msg}]" if msg else ""))


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream):
    """``stream`` (None: the current one) is the current stream within.  Tensors
    made there belong to it, as the call that fills them does (memory of another
    stream's may still be in use there), and so does what a callback launches."""
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _host(a, dtype) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=dtype))


def _shape(B: int, d: int, V: int, e_dtype: int = E_BF16, L: int = 256) -> _Shape:
    return _Shape(B, L, d, V, e_dtype)


def workspace_size(B: int, d: int, V: int, e_dtype: int = E_BF16, L: int = 256) -> int:
    """Bytes of workspace one step needs on the current device (0 if invalid)."""
    return int(lib().dg_workspace_size(ctypes.byref(_shape(B, d, V, e_dtype, L))))


def selfcond_workspace_size(B: int, d: int, V: int, e_dtype: int = E_BF16, L: int = 256) -> int:
    """Bytes of workspace a step with the self-conditioning signal needs."""
    return int(lib().dg_selfcond_workspace_size(ctypes.byref(_shape(B, d, V, e_dtype, L))))


class Workspace:
    """Device scratch for steps of one shape (a zeroed torch uint8 buffer);
    ``selfcond=True`` sizes it for ``denoise_step_selfcond``."""

    def __init__(self, B: int, d: int, V: int, e_dtype: int = E_BF16, device=None, stream=None,
                 selfcond: bool = False):
        import torch
        n = selfcond_workspace_size(B, d, V, e_dtype) if selfcond else workspace_size(B, d, V, e_dtype)
        if n == 0:
            raise DGError(2, "workspace_size")
        self.nbytes = n
        with _on(stream):
            self.buf = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
        _check(lib().dg_workspace_init(_ptr(self.buf), ctypes.c_size_t(n), _stream(stream)),
               "dg_workspace_init")


def _step_call(fn_name, h, E, step_idx, has_prev, canvas, prev_argmax, accept, entropy, sampled,
               argmax, stop, ws: Workspace, params: Params, e_scale=None, active=None, logits=None,
               stream=None):
    B = int(len(step_idx))
    R, d = h.shape
    V = E.shape[0]
    e_dtype = E_BF16 if e_scale is None else E_FP8_E4M3
    shp = _shape(B, d, V, e_dtype, L=R // max(B, 1))
    prm = params.c()
    ks = _host(step_idx, np.int32)
    hp = _host(has_prev, np.uint8)
    act = None if active is None else _host(active, np.uint8)
    args = [ctypes.byref(shp), ctypes.byref(prm), _ptr(h), _ptr(E), _ptr(e_scale),
            ks.ctypes.data_as(ctypes.c_void_p), hp.ctypes.data_as(ctypes.c_void_p),
            None if act is None else act.ctypes.data_as(ctypes.c_void_p),
            _ptr(canvas), _ptr(prev_argmax), _ptr(accept), _ptr(entropy), _ptr(sampled),
            _ptr(argmax), _ptr(stop)]
    if fn_name == "dg_debug_logits":
        args.append(_ptr(logits))
    args += [_ptr(ws.buf), ctypes.c_size_t(ws.nbytes), _stream(stream)]
    _check(getattr(lib(), fn_name)(*args), fn_name)


def denoise_step(h, E, step_idx, has_prev, canvas, prev_argmax, accept, entropy, sampled, argmax,
                 stop, ws: Workspace, params: Params = Params(), e_scale=None, active=None,
                 stream=None) -> None:
    """Enqueue one step (see ``dg_denoise_step`` in include/dg.h).

    Tensors are CUDA tensors: h bf16 [B*256, d], E bf16 [V, d] (or uint8
    E4M3 codes with ``e_scale`` float [V]), canvas / prev_argmax / sampled /
    argmax int32 [B*256], accept uint8 [B*256], entropy float32 [B*256],
    stop int32 [B].  ``step_idx``, ``has_prev`` and ``active`` are host
    sequences of length B."""
    _step_call("dg_denoise_step", h, E, step_idx, has_prev, canvas, prev_argmax, accept, entropy,
               sampled, argmax, stop, ws, params, e_scale, active, None, stream)


def denoise_step_noalloc(h, E, step_idx, has_prev, canvas, prev_argmax, accept, entropy, sampled,
                         argmax, stop, params: Params = Params(), e_scale=None, active=None,
                         stream=None) -> None:
    """``dg_denoise_step_noalloc``: the same step without a caller workspace,
    for callers that cannot allocate device memory (the scratch is a fixed
    8 MiB array inside the library; calls must not overlap on the GPU; a
    device-side fault is reported by ``noalloc_status``)."""
    B = int(len(step_idx))
    R, d = h.shape
    V = E.shape[0]
    e_dtype = E_BF16 if e_scale is None else E_FP8_E4M3
    shp = _shape(B, d, V, e_dtype, L=R // max(B, 1))
    prm = params.c()
    ks = _host(step_idx, np.int32)
    hp = _host(has_prev, np.uint8)
    act = None if active is None else _host(active, np.uint8)
    _check(lib().dg_denoise_step_noalloc(
        ctypes.byref(shp), ctypes.byref(prm), _ptr(h), _ptr(E), _ptr(e_scale),
        ks.ctypes.data_as(ctypes.c_void_p), hp.ctypes.data_as(ctypes.c_void_p),
        None if act is None else act.ctypes.data_as(ctypes.c_void_p),
        _ptr(canvas), _ptr(prev_argmax), _ptr(accept), _ptr(entropy), _ptr(sampled),
        _ptr(argmax), _ptr(stop), _stream(stream)), "dg_denoise_step_noalloc")


def noalloc_status(stream=None) -> int:
    """Synchronise and read/clear the fault latch of the allocation-free
    step's scratch array on the current device (0 = no fault)."""
    return int(lib().dg_noalloc_status(_stream(stream)))


def noalloc_selftest_bounded_wait(limit_ns: int, stream=None) -> int:
    """The bounded-wait self test against the allocation-free step's latch;
    returns the status it leaves (6 = timed out as designed)."""
    return int(lib().dg_noalloc_selftest_bounded_wait(ctypes.c_uint64(limit_ns), _stream(stream)))


def debug_logits(h, E, step_idx, has_prev, canvas, prev_argmax, accept, entropy, sampled, argmax,
                 stop, logits, ws: Workspace, params: Params = Params(), e_scale=None, active=None,
                 stream=None) -> None:
    """The same step, also writing the float32 logits [B*256, V] it consumed."""
    _step_call("dg_debug_logits", h, E, step_idx, has_prev, canvas, prev_argmax, accept, entropy,
               sampled, argmax, stop, ws, params, e_scale, active, logits, stream)


def device_status(ws: Workspace, stream=None) -> int:
    """Synchronise and read/clear the device fault latch (0 = clean)."""
    return int(lib().dg_device_status(_ptr(ws.buf), ctypes.c_size_t(ws.nbytes), _stream(stream)))


def denoise_loop(E, hidden_fn, h_buf, canvas, prev_argmax, has_prev, accept, entropy, sampled,
                 argmax, stop, ws: Workspace, params: Params = Params(), k_start: int = 0,
                 e_scale=None, stream=None):
    """Run the adaptive loop (``dg_denoise_loop``).

    ``hidden_fn(k, canvas_tensor, h_buf)`` must fill ``h_buf`` for step k on
    the current stream (``stream``, if one is given) and return None.  ``has_prev`` is a host uint8 numpy
    array [B] updated in place.  Returns the host int32 array of steps taken.
    """
    B = int(len(has_prev))
    R, d = h_buf.shape
    V = E.shape[0]
    e_dtype = E_BF16 if e_scale is None else E_FP8_E4M3
    shp = _shape(B, d, V, e_dtype, L=R // B)
    prm = params.c()
    steps = np.zeros(B, np.int32)
    assert isinstance(has_prev, np.ndarray) and has_prev.dtype == np.uint8
    errors = []

    def cb(k, canvas_ptr, h_ptr, user, stream_ptr):
        try:
            hidden_fn(int(k), canvas, h_buf)
            return 0
        except Exception as exc:  # reported as DG_ERR_CALLBACK
            errors.append(exc)
            return 1

    cfn = _HIDDEN_FN(cb)
    with _on(stream):
        code = lib().dg_denoise_loop(
            ctypes.byref(shp), ctypes.byref(prm), _ptr(E), _ptr(e_scale), cfn, None,
            ctypes.c_int32(k_start), _ptr(h_buf), _ptr(canvas), _ptr(prev_argmax),
            has_prev.ctypes.data_as(ctypes.c_void_p), steps.ctypes.data_as(ctypes.c_void_p),
            _ptr(accept), _ptr(entropy), _ptr(sampled), _ptr(argmax), _ptr(stop), _ptr(ws.buf),
            ctypes.c_size_t(ws.nbytes), _stream(stream))
    if code != 0:
        err = DGError(code, "dg_denoise_loop")
        if errors:
            raise err from errors[0]
        raise err
    return steps


def loop_state_bytes(B: int) -> int:
    """Bytes of device loop state ``dg_denoise_loop_graph`` needs for B canvases."""
    return int(lib().dg_loop_state_bytes(ctypes.c_int32(B)))


class LoopState:
    """Device loop state of the device-side loop (a torch uint8 buffer);
    ``k`` is a one-element int32 view of the step index the loop's graph
    body is about to run, for a hidden-state graph to read."""

    def __init__(self, B: int, device=None):
        import torch
        n = loop_state_bytes(B)
        if n == 0:
            raise DGError(1, "loop_state_bytes")
        self.nbytes = n
        self.buf = torch.zeros(n, dtype=torch.uint8, device=device or "cuda")
        self.k = self.buf[:4].view(torch.int32)


def denoise_loop_graph(E, hidden_graph, h_buf, canvas, prev_argmax, has_prev, accept, entropy, sampled,
                       argmax, stop, ws: Workspace, state: LoopState, params: Params = Params(),
                       k_start: int = 0, e_scale=None, stream=None):
    """The adaptive loop run on the device (``dg_denoise_loop_graph``).

    ``hidden_graph`` is a ``torch.cuda.CUDAGraph`` captured with
    ``keep_graph=True`` that writes step ``state.k``'s hidden states into
    ``h_buf`` (or None: ``h_buf`` stays as it is).  ``has_prev`` is a host
    uint8 numpy array [B] updated in place.  Returns the host int32 array of
    steps taken."""
    B = int(len(has_prev))
    R, d = h_buf.shape
    V = E.shape[0]
    e_dtype = E_BF16 if e_scale is None else E_FP8_E4M3
    shp = _shape(B, d, V, e_dtype, L=R // B)
    prm = params.c()
    steps = np.zeros(B, np.int32)
    assert isinstance(has_prev, np.ndarray) and has_prev.dtype == np.uint8
    g = None if hidden_graph is None else ctypes.c_void_p(int(hidden_graph.raw_cuda_graph()))
    _check(lib().dg_denoise_loop_graph(
        ctypes.byref(shp), ctypes.byref(prm), _ptr(E), _ptr(e_scale), g, ctypes.c_int32(k_start), _ptr(h_buf),
        _ptr(canvas), _ptr(prev_argmax), has_prev.ctypes.data_as(ctypes.c_void_p),
        steps.ctypes.data_as(ctypes.c_void_p), _ptr(accept), _ptr(entropy), _ptr(sampled), _ptr(argmax),
        _ptr(stop), _ptr(state.buf), ctypes.c_size_t(state.nbytes), _ptr(ws.buf), ctypes.c_size_t(ws.nbytes),
        _stream(stream)), "dg_denoise_loop_graph")
    return steps


class LoopGraph:
    """The device-side loop built once and run many times
    (``dg_loop_graph_create`` / ``_run`` / ``_destroy``): the buffers are
    fixed at construction (they must outlive the object); ``run`` takes the
    first step, the host uint8 ``has_prev`` array (updated in place) and
    returns the host int32 array of steps taken."""

    def __init__(self, E, hidden_graph, h_buf, canvas, prev_argmax, accept, entropy, sampled, argmax, stop,
                 ws: Workspace, state: LoopState, params: Params = Params(), e_scale=None):
        B = int(stop.shape[0])
        R, d = h_buf.shape
        V = E.shape[0]
        e_dtype = E_BF16 if e_scale is None else E_FP8_E4M3
        self.B = B
        shp = _shape(B, d, V, e_dtype, L=R // B)
        prm = params.c()
        g = None if hidden_graph is None else ctypes.c_void_p(int(hidden_graph.raw_cuda_graph()))
        handle = ctypes.c_void_p()
        # the buffers stay referenced for the handle's lifetime
        self._keep = (E, e_scale, h_buf, canvas, prev_argmax, accept, entropy, sampled, argmax, stop, ws, state)
        self._h = None
        _check(lib().dg_loop_graph_create(
            ctypes.byref(shp), ctypes.byref(prm), _ptr(E), _ptr(e_scale), g, _ptr(h_buf), _ptr(canvas),
            _ptr(prev_argmax), _ptr(accept), _ptr(entropy), _ptr(sampled), _ptr(argmax), _ptr(stop),
            _ptr(state.buf), ctypes.c_size_t(state.nbytes), _ptr(ws.buf), ctypes.c_size_t(ws.nbytes),
            ctypes.byref(handle)), "dg_loop_graph_create")
        self._h = handle

    def run(self, has_prev, k_start: int = 0, stream=None):
        assert isinstance(has_prev, np.ndarray) and has_prev.dtype == np.uint8 and len(has_prev) == self.B
        steps = np.zeros(self.B, np.int32)
        _check(lib().dg_loop_graph_run(self._h, ctypes.c_int32(k_start), has_prev.ctypes.data_as(ctypes.c_void_p),
                                       steps.ctypes.data_as(ctypes.c_void_p), _stream(stream)), "dg_loop_graph_run")
        return steps

    def close(self) -> None:
        if self._h is not None:
            lib().dg_loop_graph_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def embedder_transpose(E, E_t, e_fp8: bool = False, stream=None) -> None:
    """E_t [d, V] bf16 = E^T (``dg_embedder_transpose``); E bf16 [V, d], or
    E4M3 codes (uint8) with ``e_fp8``."""
    V, d = E.shape
    shp = _shape(1, d, V, E_FP8_E4M3 if e_fp8 else E_BF16)
    _check(lib().dg_embedder_transpose(ctypes.byref(shp), _ptr(E), _ptr(E_t), _stream(stream)),
           "dg_embedder_transpose")


def denoise_step_selfcond(h, E, E_t, step_idx, has_prev, canvas, prev_argmax, accept, entropy, sampled, argmax,
                          stop, signal, ws: Workspace, params: Params = Params(), e_scale=None,
                          stream=None) -> None:
    """One step plus the self-conditioning signal (``dg_denoise_step_selfcond``):
    ``signal`` float32 [B*256, d]; ``ws`` made with ``selfcond=True``."""
    B = int(len(step_idx))
    R, d = h.shape
    V = E.shape[0]
    e_dtype = E_BF16 if e_scale is None else E_FP8_E4M3
    shp = _shape(B, d, V, e_dtype, L=R // max(B, 1))
    prm = params.c()
    ks = _host(step_idx, np.int32)
    hp = _host(has_prev, np.uint8)
    _check(lib().dg_denoise_step_selfcond(
        ctypes.byref(shp), ctypes.byref(prm), _ptr(h), _ptr(E), _ptr(e_scale), _ptr(E_t),
        ks.ctypes.data_as(ctypes.c_void_p), hp.ctypes.data_as(ctypes.c_void_p), _ptr(canvas), _ptr(prev_argmax),
        _ptr(accept), _ptr(entropy), _ptr(sampled), _ptr(argmax), _ptr(stop), _ptr(signal), _ptr(ws.buf),
        ctypes.c_size_t(ws.nbytes), _stream(stream)), "dg_denoise_step_selfcond")


def init_canvas(canvas, B: int, V: int, params: Params = Params(), d: int = 64, stream=None) -> None:
    """Fill ``canvas`` (int32 CUDA tensor [B*256]) with the uniform noise
    block ``params.block`` starts from (``dg_init_canvas``)."""
    shp = _shape(B, d, V, E_BF16, L=int(canvas.numel()) // max(B, 1))
    prm = params.c()
    _check(lib().dg_init_canvas(ctypes.byref(shp), ctypes.byref(prm), _ptr(canvas), _stream(stream)),
           "dg_init_canvas")


def generate_blocks(E, hidden_fn, n_blocks: int, h_buf, blocks, canvas, prev_argmax, accept, entropy, sampled,
                    argmax, stop, ws: Workspace, params: Params = Params(), e_scale=None, stream=None):
    """Block-by-block generation (``dg_generate_blocks``).

    ``hidden_fn(j, k, canvas_tensor, committed, h_buf)`` fills ``h_buf``
    for step k of block j on the current stream (``stream``, if one is given);
    ``committed`` is the view
    ``blocks[:j]`` of the blocks committed so far.  ``blocks`` is an int32
    CUDA tensor [n_blocks, B*256].  Returns the host int32 array of steps
    taken, [n_blocks, B]."""
    return _run_blocks(None, E, hidden_fn, n_blocks, h_buf, blocks, canvas, prev_argmax, accept, entropy, sampled,
                       argmax, stop, ws, params, e_scale, stream)


def generate_blocks_context(plan: ContextPlan, E, hidden_fn, n_blocks: int, h_buf, blocks, canvas, prev_argmax,
                            accept, entropy, sampled, argmax, stop, ws: Workspace, params: Params = Params(),
                            e_scale=None, stream=None):
    """``generate_blocks`` with a context (``dg_generate_blocks_context``):
    ``plan`` holds the tables of the block's provisional rows whenever
    ``hidden_fn`` is called, for ``context_append`` and
    ``context_attention``; the batch it held before the call is committed
    first.  After block j's last step ``hidden_fn(j, params.max_steps, canvas,
    committed, h_buf)`` is called once more, with the finished canvas, to encode
    it: what it appends then is what the next plan commits (``h_buf`` is not
    read).  DGError 10 when a block does not fit, 9 when a key or value that is
    not finite was appended; a block that was not finished is dropped from the
    context."""
    import torch
    given = dict(E=E, h_buf=h_buf, blocks=blocks, canvas=canvas, prev_argmax=prev_argmax, accept=accept, entropy=entropy,
                 sampled=sampled, argmax=argmax, stop=stop, workspace=ws.buf, e_scale=e_scale)
    for name, t in given.items():
        _need(t is None or t.device == plan.device, f"{name} is on another device than the plan, {plan.device}")
    _need(stream is None or stream.device == plan.device, "the stream belongs to another device than the plan")
    with torch.cuda.device(plan.device):
        return _run_blocks(plan, E, hidden_fn, n_blocks, h_buf, blocks, canvas, prev_argmax, accept, entropy, sampled,
                           argmax, stop, ws, params, e_scale, stream)


def _run_blocks(plan, E, hidden_fn, n_blocks, h_buf, blocks, canvas, prev_argmax, accept, entropy, sampled, argmax,
                stop, ws, params, e_scale, stream):
    R, d = h_buf.shape
    B = int(len(stop))
    V = E.shape[0]
    e_dtype = E_BF16 if e_scale is None else E_FP8_E4M3
    shp = _shape(B, d, V, e_dtype, L=R // B)
    prm = params.c()
    steps = np.zeros((n_blocks, B), np.int32)
    errors = []

    def cb(j, k, canvas_ptr, committed_ptr, h_ptr, user, stream_ptr):
        try:
            hidden_fn(int(j), int(k), canvas, blocks[:int(j)], h_buf)
            return 0
        except Exception as exc:  # reported as DG_ERR_CALLBACK
            errors.append(exc)
            return 1

    cfn = _BLOCK_HIDDEN_FN(cb)
    head = (ctypes.byref(shp), ctypes.byref(prm), _ptr(E), _ptr(e_scale), ctypes.c_int32(n_blocks), cfn, None)
    tail = (_ptr(h_buf), _ptr(blocks), steps.ctypes.data_as(ctypes.c_void_p), _ptr(canvas), _ptr(prev_argmax),
            _ptr(accept), _ptr(entropy), _ptr(sampled), _ptr(argmax), _ptr(stop), _ptr(ws.buf),
            ctypes.c_size_t(ws.nbytes), _stream(stream))
    with _on(stream):
        if plan is None:
            where = "dg_generate_blocks"
            code = lib().dg_generate_blocks(*head, *tail)
        else:
            where = "dg_generate_blocks_context"
            code = lib().dg_generate_blocks_context(*head, plan._ref, _ptr(plan.add), *tail)
    if code != 0:
        err = DGError(code, where)
        if errors:
            raise err from errors[0]
        raise err
    return steps


# ---------------------------------------------------------------------------
# the context of block-by-block generation: block tables, rotary positions,
# the 8-bit paged cache and the attention over it
# ---------------------------------------------------------------------------

PAGE = 64  # token slots per page

_plans = itertools.count()

_ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise DGError(1, what)


def _need_int32(**sizes) -> None:
    """ctypes would take the low 32 bits of a number that is too large."""
    for name, n in sizes.items():
        _need(-2 ** 31 <= n < 2 ** 31, f"{name} = {n} is beyond 32 bits")


def _call(device, fn, where, stream, *args):
    """Call a library function on ``stream`` (None: the current one) with the
    tensors' device current."""
    import torch
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device.index)
    else:
        _need(stream.device == device, "the stream belongs to another device than the tensors")
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        code = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            code = fn(*args, handle)
    if code != 0:
        _check(code, where)


def _heads(t, rows, heads, dim, device, name) -> _Heads:
    import torch
    if t.dtype is not torch.bfloat16 or t.dim() != 3 or t.device != device:
        raise DGError(1, f"{name} must be a bfloat16 tensor [rows, heads, dim] on {device}")
    n, h, d = t.shape
    rs, hs, ds = t.stride()
    if n < rows or h != heads or d != dim:
        raise DGError(2, f"{name} must be [{rows} (or more), {heads}, {dim}], not {list(t.shape)}")
    # the stride of a dimension of one element is not a property of the data
    if h == 1:
        hs = dim
    if n == 1:
        rs = max(rs if rs % 8 == 0 else 0, dim)
    ptr = t.data_ptr()
    if ds != 1 or rs < dim or (h > 1 and hs < dim) or rs % 8 or hs % 8 or ptr % 16:
        raise DGError(1, f"{name} needs contiguous heads, strides of multiples of 8 elements and 16-byte alignment")
    return _Heads(ptr, rs, hs)


class ContextPlan:
    """The state of a context and the tables of its provisional batch
    (``dg_context`` in include/dg.h), as int32 CUDA tensors (``slots`` int64):
    ``table`` [B, max_pages], ``held`` [B], ``free_list`` [pages],
    ``free_count`` [1]; results ``lens`` [B], ``start`` [B + 1], ``positions``
    and ``slots`` [rows], ``runs`` [rows // 64 + 2 B, 4], ``free_next`` [1],
    ``status`` [2], ``epoch`` [1].  A new plan is empty, all pages free."""

    def __init__(self, B: int, rows: int, pages: int, max_pages: int, device=None):
        import torch
        _need(min(B, rows, pages, max_pages) >= 1, "ContextPlan sizes must be positive")
        _need_int32(B=B, rows=rows, pages=pages, max_pages=max_pages)
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.B, self.rows, self.pages, self.max_pages, self.device = int(B), int(rows), int(pages), int(max_pages), device

        def zeros(*n, dtype=torch.int32):
            return torch.zeros(n, dtype=dtype, device=device)
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32, device=device)
        self.held, self.lens, self.start = zeros(B), zeros(B), zeros(B + 1)
        self.free_list = torch.arange(pages, dtype=torch.int32, device=device)
        self.free_count, self.free_next = zeros(1) + pages, zeros(1) + pages
        self.positions, self.slots = zeros(rows) - 1, zeros(rows, dtype=torch.int64) - 1
        self.runs = zeros(rows // PAGE + 2 * B, 4)
        self.runs[:, 0] = -1
        self.status = zeros(2)
        # plans that use one cache start far apart
        self.epoch = torch.full((1,), next(_plans) * 0x9E3779B1 % 2 ** 31, dtype=torch.int32, device=device)
        self.add = zeros(B)  # lengths of generate_blocks_context
        self._c = _Context(B, rows, pages, max_pages, *(getattr(self, n).data_ptr() for n in (
            "table", "held", "free_list", "free_count", "lens", "start", "positions", "slots", "runs", "free_next",
            "status", "epoch")))
        self._ref = ctypes.byref(self._c)


def context_plan(plan: ContextPlan, add, release=None, commit: bool = False, stream=None) -> None:
    """Plan a batch (``dg_context_plan``): request r adds ``add[r]`` tokens
    (int32 CUDA tensor [B]).  ``release``: uint8 or bool CUDA tensor [B] of
    requests that leave first.  ``commit``: the batch before becomes part of
    the context; otherwise it is planned over."""
    import torch
    _need(add.dtype == torch.int32 and add.shape == (plan.B,) and add.is_contiguous() and add.device == plan.device,
          "add must be a contiguous int32 tensor [B] on the plan's device")
    _need(release is None or (release.dtype in (torch.uint8, torch.bool) and release.shape == (plan.B,) and
                              release.is_contiguous() and release.device == plan.device),
          "release must be a contiguous uint8 tensor [B] on the plan's device")
    _call(plan.device, lib().dg_context_plan, "dg_context_plan", stream, plan._ref, add.data_ptr(),
          None if release is None else release.data_ptr(), 1 if commit else 0)


def context_status(plan: ContextPlan, stream=None) -> int:
    """Synchronise and report (``dg_context_status``): 10 (the last batch was
    refused), else 9 (an append met a value that is not finite; cleared by this
    answer), else 0."""
    import torch
    with torch.cuda.device(plan.device):
        return int(lib().dg_context_status(plan._ref, _stream(stream)))


class RopeFrequencies:
    """Rotary frequencies on the device (``dg_rope_frequencies``): ``rot``
    elements of each head turn; ``scaling`` "none", "linear", "ntk" or
    "parts" by ``factor`` beyond ``original_length`` positions."""

    def __init__(self, rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 original_length: int = 4096, interleaved: bool = False, device=None):
        import torch
        _need(scaling in _ROPE_SCALING, f"scaling must be one of {sorted(_ROPE_SCALING)}")
        _need_int32(rot=rot, original_length=original_length)
        f = np.zeros(max(int(rot), 2) // 2, np.float64)
        mag = ctypes.c_float()
        _check(lib().dg_rope_frequencies(rot, base, _ROPE_SCALING[scaling], factor, original_length,
                                         f.ctypes.data_as(ctypes.c_void_p), ctypes.byref(mag)), "dg_rope_frequencies")
        self.rot, self.interleaved, self.magnitude = int(rot), bool(interleaved), float(mag.value)
        self.freq = torch.from_numpy(f).to("cuda" if device is None else device)
        self._c = _RopeArgs(self.rot, int(self.interleaved), self.magnitude, self.freq.data_ptr())
        self._ref = ctypes.byref(self._c)


def rope(x, positions, frequencies: RopeFrequencies, out=None, stream=None):
    """Rotary positions (``dg_rope``): bfloat16 ``x`` [rows, heads, dim], int32
    ``positions`` [rows]; returns ``out`` (``x`` itself for in place).  None: a new
    tensor, one of ``stream``'s, whose rows without a position are 0."""
    import torch
    if out is None:
        _need(stream is None or stream.device == x.device, "the stream belongs to another device than the tensors")
        with _on(stream):
            out = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
    _need(x.dim() == 3, "x must be [rows, heads, dim]")
    rows, heads, dim = x.shape
    _need(positions.dtype == torch.int32 and positions.dim() == 1 and positions.is_contiguous() and
          positions.numel() >= rows and positions.device == x.device == frequencies.freq.device,
          "positions must be a contiguous int32 tensor [rows] on x's device, and so the frequencies")
    _need(out.shape == x.shape, "out must have x's shape")
    if rows == 0:
        return out
    a, b = _heads(x, rows, heads, dim, x.device, "x"), _heads(out, rows, heads, dim, x.device, "out")
    _call(x.device, lib().dg_rope, "dg_rope", stream, ctypes.byref(a), ctypes.byref(b), rows, heads, dim,
          positions.data_ptr(), frequencies._ref)
    return out


class ContextCache:
    """One layer's cache (``dg_context_cache``): E4M3 codes ``k``, ``v`` (uint8
    [pages, heads, 64, dim]) and power-of-two scales ``k_scale``, ``v_scale``
    (float32 [pages, heads]); ``kept``: held tokens' codes as they were before a
    provisional batch, which ``context_append`` keeps for itself (one page a
    request, 256 at most)."""

    def __init__(self, pages: int, heads: int, dim: int, device=None):
        import torch
        device = "cuda" if device is None else device
        _need(min(pages, heads, dim) >= 1, "ContextCache sizes must be positive")
        _need_int32(pages=pages, heads=heads, dim=dim)
        self.pages, self.heads, self.dim = int(pages), int(heads), int(dim)
        self.k = torch.zeros((pages, heads, PAGE, dim), dtype=torch.uint8, device=device)
        self.v = torch.zeros_like(self.k)
        self.k_scale = torch.ones((pages, heads), dtype=torch.float32, device=device)
        self.v_scale = torch.ones_like(self.k_scale)
        self.kept = torch.zeros(lib().dg_context_kept_size(pages, heads, dim), dtype=torch.uint8, device=device)
        self.device = self.k.device
        self._c = _Cache(self.pages, self.heads, self.dim, self.k.data_ptr(), self.v.data_ptr(),
                         self.k_scale.data_ptr(), self.v_scale.data_ptr(), self.kept.data_ptr())
        self._ref = ctypes.byref(self._c)


def context_append(plan: ContextPlan, cache: ContextCache, k, v, rope: RopeFrequencies = None, stream=None) -> None:
    """Write the batch's keys (rotated by their positions with ``rope``) and
    values, bfloat16 [plan.rows, heads, dim], into their slots of ``cache``
    (``dg_context_append``).  Rows that take the place of a batch's (a canvas's
    next step) are best planned again first: the append then starts from the
    held tokens as they were committed."""
    dev = plan.device
    _need(cache.device == dev and (rope is None or rope.freq.device == dev),
          "the cache and the frequencies must be on the plan's device")
    a = _heads(k, plan.rows, cache.heads, cache.dim, dev, "k")
    b = _heads(v, plan.rows, cache.heads, cache.dim, dev, "v")
    _call(dev, lib().dg_context_append, "dg_context_append", stream, plan._ref, cache._ref, ctypes.byref(a),
          ctypes.byref(b), None if rope is None else rope._ref)


def context_workspace_size(rows: int, q_heads: int, kv_heads: int, dim: int) -> int:
    """Bytes of workspace ``context_attention`` needs on the current device (0 if invalid)."""
    _need_int32(rows=rows, q_heads=q_heads, kv_heads=kv_heads, dim=dim)
    return int(lib().dg_context_workspace_size(rows, q_heads, kv_heads, dim))


class ContextWorkspace:
    """Device scratch of ``context_attention`` for one shape (a zeroed torch
    uint8 buffer, one of ``stream``'s; ``device_status`` reads its fault latch)."""

    def __init__(self, rows: int, q_heads: int, kv_heads: int, dim: int, device=None, stream=None):
        import torch
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        _need(stream is None or device.index is None or stream.device == device,
              "the stream belongs to another device than the workspace")
        with torch.cuda.device(device):
            n = context_workspace_size(rows, q_heads, kv_heads, dim)
            if n == 0:
                raise DGError(2, "context_workspace_size")
            self.nbytes = n
            with _on(stream):
                self.buf = torch.empty(n, dtype=torch.uint8, device=device)
            _check(lib().dg_workspace_init(_ptr(self.buf), ctypes.c_size_t(n), _stream(stream)), "dg_workspace_init")


def context_attention(plan: ContextPlan, cache: ContextCache, q, out, ws: ContextWorkspace, causal=None,
                      window: int = 0, scale: float = None, lse=None, max_new: int = 0, stream=None) -> None:
    """Attention of the batch's rows over the cache (``dg_context_attention``):
    bfloat16 ``q``, ``out`` [plan.rows, heads, dim]; ``causal`` uint8 or bool
    CUDA tensor [B] (None: no request is causal); ``lse`` float32
    [plan.rows, heads] or None; ``max_new`` the most rows of one request, if
    known."""
    import torch
    dev = plan.device
    _need(cache.device == dev and ws.buf.device == dev, "the cache and the workspace must be on the plan's device")
    _need(q.dim() == 3, "q must be [rows, heads, dim]")
    heads = q.shape[1]
    a = _heads(q, plan.rows, heads, cache.dim, dev, "q")
    b = _heads(out, plan.rows, heads, cache.dim, dev, "out")
    _need(causal is None or (causal.dtype in (torch.uint8, torch.bool) and causal.shape == (plan.B,) and
                             causal.is_contiguous() and causal.device == dev),
          "causal must be a contiguous uint8 tensor [B] on the plan's device")
    _need(lse is None or (lse.dtype == torch.float32 and lse.dim() == 2 and lse.shape[0] >= plan.rows and
                          lse.shape[1] == heads and lse.is_contiguous() and lse.device == dev),
          "lse must be a contiguous float32 tensor [rows, heads] on the plan's device")
    _need(scale is None or np.float32(scale) > 0, "scale must be positive, in 32 bits too (0 would stand for the default)")
    _need_int32(window=window, max_new=max_new)
    _call(dev, lib().dg_context_attention, "dg_context_attention", stream, plan._ref, cache._ref, ctypes.byref(a),
          ctypes.byref(b), heads, 0.0 if scale is None else scale, None if causal is None else causal.data_ptr(),
          window, max_new, None if lse is None else lse.data_ptr(), ws.buf.data_ptr(), ws.nbytes)


def debug_gumbel(words, stream=None):
    """Device g32 and the screening pass's approximate lg2(E / ln 2), E = -ln u,
    for uint32 words (torch int32 CUDA tensor)."""
    import torch
    n = int(words.numel())
    with _on(stream):
        g = torch.empty(n, dtype=torch.float32, device=words.device)
        a = torch.empty(n, dtype=torch.float32, device=words.device)
    _check(lib().dg_debug_gumbel(_ptr(words), ctypes.c_int32(n), _ptr(g), _ptr(a), _stream(stream)),
           "dg_debug_gumbel")
    return g, a


def set_head_events(ev_start=None, ev_stop=None) -> None:
    """Record torch.cuda.Events around the fused head kernel of later steps
    on this thread (None, None clears)."""
    a = None if ev_start is None else ctypes.c_void_p(ev_start.cuda_event)
    b = None if ev_stop is None else ctypes.c_void_p(ev_stop.cuda_event)
    _check(lib().dg_set_head_events(a, b), "dg_set_head_events")


def selftest_bounded_wait(limit_ns: int, ws: Workspace, stream=None) -> int:
    """Run the bounded-wait self test; returns the status code (6 = timed out as designed)."""
    return int(lib().dg_selftest_bounded_wait(ctypes.c_uint64(limit_ns), _ptr(ws.buf),
                                              ctypes.c_size_t(ws.nbytes), _stream(stream)))


# ---------------------------------------------------------------------------
# vocabulary-sharded step (dg_head_partials / dg_merge_partials)
# ---------------------------------------------------------------------------

def partials_count(B: int, d: int, V_shard: int, e_dtype: int = E_BF16, L: int = 256) -> int:
    """Records per row that one shard's head writes (``dg_partials_count``)."""
    return int(lib().dg_partials_count(ctypes.byref(_shape(B, d, V_shard, e_dtype, L))))


def head_partials(h, E_shard, v_offset: int, step_idx, partials, ws: Workspace, params: Params = Params(),
                  e_scale=None, stream=None) -> None:
    """Head and sampler over vocabulary rows v_offset .. v_offset + len(E_shard) - 1,
    writing the float32 records [7, B*256, count] into ``partials``."""
    B = int(len(step_idx))
    R, d = h.shape
    shp = _shape(B, d, E_shard.shape[0], E_BF16 if e_scale is None else E_FP8_E4M3, L=R // max(B, 1))
    prm = params.c()
    ks = _host(step_idx, np.int32)
    _check(lib().dg_head_partials(ctypes.byref(shp), ctypes.byref(prm), ctypes.c_int32(v_offset), _ptr(h),
                                  _ptr(E_shard), _ptr(e_scale), ks.ctypes.data_as(ctypes.c_void_p),
                                  _ptr(partials), _ptr(ws.buf), ctypes.c_size_t(ws.nbytes), _stream(stream)),
           "dg_head_partials")


def merge_partials(partials, V: int, d: int, step_idx, has_prev, canvas, prev_argmax, accept, entropy, sampled,
                   argmax, stop, ws: Workspace, params: Params = Params(), active=None, stream=None) -> None:
    """Merge the gathered records ``partials`` [S, 7, B*256, count] over the
    whole vocabulary V, then selection, renoise and stop."""
    B = int(len(step_idx))
    S, _, R, count = partials.shape
    shp = _shape(B, d, V, E_BF16, L=R // max(B, 1))
    prm = params.c()
    ks = _host(step_idx, np.int32)
    hp = _host(has_prev, np.uint8)
    act = None if active is None else _host(active, np.uint8)
    _check(lib().dg_merge_partials(ctypes.byref(shp), ctypes.byref(prm), _ptr(partials), ctypes.c_int32(S),
                                   ctypes.c_int32(count), ks.ctypes.data_as(ctypes.c_void_p),
                                   hp.ctypes.data_as(ctypes.c_void_p),
                                   None if act is None else act.ctypes.data_as(ctypes.c_void_p),
                                   _ptr(canvas), _ptr(prev_argmax), _ptr(accept), _ptr(entropy), _ptr(sampled),
                                   _ptr(argmax), _ptr(stop), _ptr(ws.buf), ctypes.c_size_t(ws.nbytes),
                                   _stream(stream)), "dg_merge_partials")


def gather_partials(local, group=None):
    """All-gather one rank's records [7, R, count] into [world, 7, R, count]
    (torch.distributed over the default or given process group; NCCL for
    CUDA tensors).  The only collective of the sharded step."""
    import torch
    import torch.distributed as dist
    world = dist.get_world_size(group)
    local = local.contiguous()
    out = torch.empty((world * local.shape[0],) + tuple(local.shape[1:]), dtype=local.dtype, device=local.device)
    dist.all_gather_into_tensor(out, local, group=group)
    return out.view((world,) + tuple(local.shape))
