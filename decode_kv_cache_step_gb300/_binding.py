"""ctypes binding of liblf_decode.so: argument marshalling only.

Every function here validates torch tensors (dtype, device, shape, layout),
passes their data pointers and the stream to the C ABI declared in
``include/lf_decode.h`` and raises ``LFError`` on a non-OK status. All of the
decode step's arithmetic runs in the library's CUDA kernels; there is no CPU
or PyTorch fallback, and a missing library is an error.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import os
import threading

import torch

from . import build as _build

LF_OK = 0
LF_ERR_INVALID_ARG = 1
LF_ERR_UNSUPPORTED = 2
LF_ERR_CUDA = 3
LF_ERR_NO_MEMORY = 4

LF_DEVERR_BAD_WRITE_SLOT = 0x1
LF_DEVERR_WAIT_TIMEOUT = 0x2
LF_DEVERR_BAD_LENGTH = 0x4

LF_KERNEL_DECODE_STEP = 0
LF_KERNEL_ATTENTION = 1
LF_KERNEL_SCORE = 2
LF_KERNEL_NORM_ROPE = 3
LF_KERNEL_PACKED_ATTENTION = 4
LF_KERNEL_KV4 = 5
LF_KERNEL_PROMPT_WEIGHTS = 6
KERNEL_NAMES = {LF_KERNEL_DECODE_STEP: "lf_decode_step_kernel",
                LF_KERNEL_ATTENTION: "lf_decode_step_kernel (attention-only variant)",
                LF_KERNEL_SCORE: "lf_score_kernel",
                LF_KERNEL_NORM_ROPE: "lf_rope_kernel",
                LF_KERNEL_PACKED_ATTENTION: "lf_attn_kernel",
                LF_KERNEL_KV4: "lf_kv4_pack_kernel, lf_kv4_unpack_kernel, lf_kv4_attn_kernel",
                LF_KERNEL_PROMPT_WEIGHTS: "lf_prompt_weights_kernel"}

LF_STEP_FILL_EMPTY_FIRST = 0x1
LF_STEP_MASK_EVICTED = 0x2
LF_STEP_LOG2_SCORES = 0x4
LF_MAX_TOPK = 1024
LF_MAX_AXES = 4

# Every exported symbol of include/lf_decode.h.
EXPORTED = (
    "lf_decode_step", "lf_decode_step_scores", "lf_decode_step_ex", "lf_decode_attention",
    "lf_decode_step_host", "lf_decode_step_noalloc", "lf_step_prepare", "lf_step_run",
    "lf_step_errors", "lf_step_destroy", "lf_step_plan", "lf_device_errors",
    "lf_qk_norm_rope", "lf_prefill_append", "lf_window_attention",
    "lf_window_attention_workspace", "lf_decode_step_prefix", "lf_decode_attention_prefix",
    "lf_decode_prefix_workspace",
    "lf_qk_norm_rope_axes", "lf_prefill_append_axes", "lf_decode_step_weights",
    "lf_decode_weights_workspace", "lf_prompt_weights", "lf_prompt_weights_workspace",
    "lf_kv4_pack", "lf_kv4_unpack", "lf_decode_attention_kv4", "lf_decode_kv4_workspace",
    "lf_profile_enable", "lf_profile_collect", "lf_release_workspace", "lf_status_string",
    "lf_last_error", "lf_version",
)


class LFError(RuntimeError):
    """A non-OK lf_status from the library."""

    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load_library(path: str | None = None):
    """Load (once) and bind the shared library. Raises if it is missing.

    The environment variable LF_LIBRARY names another build of the same
    library (for comparing two builds in one session)."""
    global _lib, _fast_pointers
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or os.environ.get("LF_LIBRARY") or _build.LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"{p} is missing: build it first with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(p)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        step_args = [P] * 9 + [I] * 6 + [F, P]
        lib.lf_decode_step.argtypes = step_args
        lib.lf_decode_step_host.argtypes = step_args
        lib.lf_decode_step_noalloc.argtypes = step_args
        lib.lf_decode_step_noalloc.restype = I
        lib.lf_decode_step_scores.argtypes = [P] * 10 + [I] * 6 + [F, P]
        lib.lf_decode_step_ex.argtypes = [P] * 9 + [I, I, P] + [I] * 6 + [F, P]
        lib.lf_decode_step_ex.restype = I
        lib.lf_decode_attention.argtypes = [P] * 8 + [I] * 5 + [F, P]
        lib.lf_decode_attention.restype = I
        for fn in (lib.lf_decode_step, lib.lf_decode_step_host, lib.lf_decode_step_scores):
            fn.restype = I
        lib.lf_step_prepare.argtypes = [P] * 9 + [I] * 6 + [F, P, ctypes.POINTER(P)]
        lib.lf_step_prepare.restype = I
        lib.lf_step_run.argtypes = [P]
        lib.lf_step_run.restype = I
        lib.lf_step_errors.argtypes = [P, ctypes.POINTER(ctypes.c_uint32), I]
        lib.lf_step_errors.restype = I
        lib.lf_step_destroy.argtypes = [P]
        lib.lf_step_destroy.restype = I
        lib.lf_step_plan.argtypes = [I] * 6 + [ctypes.POINTER(ctypes.c_int32)]
        lib.lf_step_plan.restype = I
        L, Z = ctypes.c_int64, ctypes.c_size_t
        lib.lf_qk_norm_rope.argtypes = [P, L] + [P] * 7 + [I] * 6 + [F, P]
        lib.lf_prefill_append.argtypes = [P, L] + [P] * 10 + [I] * 8 + [F, P]
        lib.lf_window_attention.argtypes = [P] * 6 + [I] * 8 + [F, P, Z, P]
        lib.lf_window_attention_workspace.argtypes = [I] * 8 + [ctypes.POINTER(Z)]
        lib.lf_decode_step_prefix.argtypes = [P] * 13 + [I, I, P] + [I] * 8 + [F, P, Z, P]
        lib.lf_decode_attention_prefix.argtypes = [P] * 12 + [I] * 7 + [F, P, Z, P]
        lib.lf_decode_prefix_workspace.argtypes = [I] * 7 + [ctypes.POINTER(Z)]
        lib.lf_qk_norm_rope_axes.argtypes = [P, L] + [P] * 4 + [ctypes.c_char_p, I] + [P] * 3 + [I] * 6 + [F, P]
        lib.lf_prefill_append_axes.argtypes = ([P, L] + [P] * 6 + [ctypes.c_char_p, I] + [P] * 4
                                               + [I] * 8 + [F, P])
        lib.lf_decode_step_weights.argtypes = [P] * 10 + [I] * 8 + [F, F, P, Z, P]
        lib.lf_decode_weights_workspace.argtypes = [I] * 6 + [ctypes.POINTER(Z)]
        lib.lf_prompt_weights.argtypes = [P] * 5 + [I] * 7 + [F, P, Z, P]
        lib.lf_prompt_weights_workspace.argtypes = [I] * 7 + [ctypes.POINTER(Z)]
        lib.lf_kv4_pack.argtypes = [P] * 9 + [I] * 5 + [P]
        lib.lf_kv4_unpack.argtypes = [P] * 8 + [I] * 5 + [P]
        lib.lf_decode_attention_kv4.argtypes = [P] * 10 + [I] * 5 + [F, P, Z, P]
        lib.lf_decode_kv4_workspace.argtypes = [I] * 5 + [ctypes.POINTER(Z)]
        for fn in (lib.lf_qk_norm_rope, lib.lf_prefill_append, lib.lf_window_attention,
                   lib.lf_window_attention_workspace, lib.lf_decode_step_prefix,
                   lib.lf_decode_attention_prefix, lib.lf_decode_prefix_workspace,
                   lib.lf_qk_norm_rope_axes, lib.lf_prefill_append_axes,
                   lib.lf_decode_step_weights, lib.lf_decode_weights_workspace,
                   lib.lf_prompt_weights, lib.lf_prompt_weights_workspace, lib.lf_kv4_pack,
                   lib.lf_kv4_unpack, lib.lf_decode_attention_kv4, lib.lf_decode_kv4_workspace):
            fn.restype = I
        lib.lf_device_errors.argtypes = [P, ctypes.POINTER(ctypes.c_uint32), I]
        lib.lf_device_errors.restype = I
        lib.lf_profile_enable.argtypes = [I]
        lib.lf_profile_enable.restype = I
        lib.lf_profile_collect.argtypes = [I, ctypes.POINTER(ctypes.c_double),
                                           ctypes.POINTER(ctypes.c_int64)]
        lib.lf_profile_collect.restype = I
        lib.lf_release_workspace.argtypes = []
        lib.lf_release_workspace.restype = I
        lib.lf_status_string.argtypes = [I]
        lib.lf_status_string.restype = ctypes.c_char_p
        lib.lf_last_error.argtypes = []
        lib.lf_last_error.restype = ctypes.c_char_p
        lib.lf_version.argtypes = []
        lib.lf_version.restype = I
        if path is None:
            _fast_pointers = _load_check()
            _lib = lib
        return lib


def _check(lib, status: int):
    if status != LF_OK:
        msg = lib.lf_last_error().decode(errors="replace")
        name = lib.lf_status_string(status).decode(errors="replace")
        raise LFError(status, f"{name}: {msg}")


def _stream_handle(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _need(t: torch.Tensor, name: str, dtype, shape, cuda: bool):
    # One combined test on the common path; the detailed ones name the fault.
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.is_cuda is cuda and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if not cuda and t.is_cuda:
        raise ValueError(f"{name}: must be a host tensor")


def _load_check():
    """lib/_lf_check.so's pointers(), None where it was not built or does not load."""
    if not os.path.exists(_build.CHECK_PATH):
        return None
    try:
        loader = importlib.machinery.ExtensionFileLoader("_lf_check", _build.CHECK_PATH)
        spec = importlib.util.spec_from_loader("_lf_check", loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
    except ImportError:  # built for another torch
        return None
    same = getattr(module, "torch_version", None) == torch.__version__
    return module.pointers if same else None


_fast_pointers = None  # (load_library sets it: importing the package maps no library)


def _pointers(*args):
    """Data pointers of tensors (None for None), given as tensor, name, dtype, shape
    each: contiguous CUDA tensors on one device, or an error that names the fault."""
    if _fast_pointers is not None:
        got = _fast_pointers(*args)
        if got is not None:
            return got
    each = [args[i:i + 4] for i in range(0, len(args), 4)]
    for t, name, dtype, shape in each:
        if t is not None:
            _need(t, name, dtype, shape, True)
    there = [t for t, _, _, _ in each if t is not None]
    for t in there:
        if t.device != there[0].device:
            raise ValueError(f"tensors on {there[0].device} and {t.device}: all must be on one device")
    return tuple(None if t is None else t.data_ptr() for t, _, _, _ in each)


def _shapes(q, k_cache):
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [B,Hq,d] and k_cache [B,Hkv,S,d]")
    B, Hq, d = q.shape
    _, Hkv, S, _ = k_cache.shape
    return int(B), int(Hq), int(Hkv), int(d), int(S)


def _check_step(q, k_cache, v_cache, mask, new_k, new_v, write_slot, out, next_slot,
                io_on_device=True, k=None):
    B, Hq, Hkv, d, S = _shapes(q, k_cache)
    bf, i32 = torch.bfloat16, torch.int32
    _need(q, "q", bf, (B, Hq, d), io_on_device)
    _need(k_cache, "k_cache", bf, (B, Hkv, S, d), True)
    _need(v_cache, "v_cache", bf, (B, Hkv, S, d), True)
    _need(mask, "mask", i32, (B, Hkv, S), True)
    _need(new_k, "new_k", bf, (B, Hkv, d), io_on_device)
    _need(new_v, "new_v", bf, (B, Hkv, d), io_on_device)
    _need(write_slot, "write_slot", i32, (B, Hkv), io_on_device)
    _need(out, "out", bf, (B, Hq, d), io_on_device)
    _need(next_slot, "next_slot", i32, (B, Hkv) if k is None else (B, Hkv, int(k)), io_on_device)
    return B, Hq, Hkv, d, S


def decode_step(q, k_cache, v_cache, mask, new_k, new_v, write_slot, out, next_slot, W, scale,
                stream=None):
    """lf_decode_step on CUDA tensors (see include/lf_decode.h). Asynchronous."""
    lib = load_library()
    B, Hq, Hkv, d, S = _check_step(q, k_cache, v_cache, mask, new_k, new_v, write_slot, out,
                                   next_slot)
    _check(lib, lib.lf_decode_step(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), mask.data_ptr(), new_k.data_ptr(),
        new_v.data_ptr(), write_slot.data_ptr(), out.data_ptr(), next_slot.data_ptr(),
        B, Hq, Hkv, d, S, int(W), float(scale), _stream_handle(stream)))


def decode_step_scores(q, k_cache, v_cache, mask, new_k, new_v, write_slot, out, next_slot,
                       scores, W, scale, stream=None):
    """lf_decode_step_scores: also fills scores [B,Hkv,S] fp32 (+inf on masked slots)."""
    lib = load_library()
    B, Hq, Hkv, d, S = _check_step(q, k_cache, v_cache, mask, new_k, new_v, write_slot, out,
                                   next_slot)
    _need(scores, "scores", torch.float32, (B, Hkv, S), True)
    _check(lib, lib.lf_decode_step_scores(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), mask.data_ptr(), new_k.data_ptr(),
        new_v.data_ptr(), write_slot.data_ptr(), out.data_ptr(), next_slot.data_ptr(),
        scores.data_ptr(), B, Hq, Hkv, d, S, int(W), float(scale), _stream_handle(stream)))


def decode_step_ex(q, k_cache, v_cache, mask, new_k, new_v, write_slot, out, next_slots, W,
                   scale, k=1, flags=0, scores=None, stream=None):
    """lf_decode_step_ex: next_slots [B,Hkv,k] int32 gets the k lowest-(score, slot)
    candidates per unit; flags are LF_STEP_* bits; scores optional [B,Hkv,S]
    (log2 I_j with LF_STEP_LOG2_SCORES)."""
    lib = load_library()
    B, Hq, Hkv, d, S = _check_step(q, k_cache, v_cache, mask, new_k, new_v, write_slot, out,
                                   next_slots, k=k)
    if scores is not None:
        _need(scores, "scores", torch.float32, (B, Hkv, S), True)
    _check(lib, lib.lf_decode_step_ex(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), mask.data_ptr(), new_k.data_ptr(),
        new_v.data_ptr(), write_slot.data_ptr(), out.data_ptr(), next_slots.data_ptr(), int(k),
        int(flags), None if scores is None else scores.data_ptr(), B, Hq, Hkv, d, S, int(W),
        float(scale), _stream_handle(stream)))


def decode_attention(q, k_cache, v_cache, mask, new_k, new_v, write_slot, out, scale,
                     stream=None):
    """lf_decode_attention: slot write and attention only (no score, no eviction)."""
    lib = load_library()
    B, Hq, Hkv, d, S = _shapes(q, k_cache)
    bf, i32 = torch.bfloat16, torch.int32
    _need(q, "q", bf, (B, Hq, d), True)
    _need(k_cache, "k_cache", bf, (B, Hkv, S, d), True)
    _need(v_cache, "v_cache", bf, (B, Hkv, S, d), True)
    _need(mask, "mask", i32, (B, Hkv, S), True)
    _need(new_k, "new_k", bf, (B, Hkv, d), True)
    _need(new_v, "new_v", bf, (B, Hkv, d), True)
    _need(write_slot, "write_slot", i32, (B, Hkv), True)
    _need(out, "out", bf, (B, Hq, d), True)
    _check(lib, lib.lf_decode_attention(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), mask.data_ptr(), new_k.data_ptr(),
        new_v.data_ptr(), write_slot.data_ptr(), out.data_ptr(), B, Hq, Hkv, d, S, float(scale),
        _stream_handle(stream)))


def decode_step_host(q, k_cache, v_cache, mask, new_k, new_v, write_slot, out, next_slot, W,
                     scale, stream=None):
    """lf_decode_step_host: per-step I/O in host tensors, caches and mask on the
    device. Pinned tensors are read and written by the kernel in place; others
    are staged through device memory. Outputs are valid after the stream syncs."""
    lib = load_library()
    B, Hq, Hkv, d, S = _check_step(q, k_cache, v_cache, mask, new_k, new_v, write_slot, out,
                                   next_slot, io_on_device=False)
    _check(lib, lib.lf_decode_step_host(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), mask.data_ptr(), new_k.data_ptr(),
        new_v.data_ptr(), write_slot.data_ptr(), out.data_ptr(), next_slot.data_ptr(),
        B, Hq, Hkv, d, S, int(W), float(scale), _stream_handle(stream)))


def decode_step_noalloc(q, k_cache, v_cache, mask, new_k, new_v, write_slot, out, next_slot, W,
                        scale, stream=None):
    """lf_decode_step_noalloc: lf_decode_step with the library's fixed 16 MiB
    scratch instead of cudaMalloc, for callers that cannot allocate device
    memory. Calls that overlap on the GPU share that scratch and race."""
    lib = load_library()
    B, Hq, Hkv, d, S = _check_step(q, k_cache, v_cache, mask, new_k, new_v, write_slot, out,
                                   next_slot)
    _check(lib, lib.lf_decode_step_noalloc(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), mask.data_ptr(), new_k.data_ptr(),
        new_v.data_ptr(), write_slot.data_ptr(), out.data_ptr(), next_slot.data_ptr(),
        B, Hq, Hkv, d, S, int(W), float(scale), _stream_handle(stream)))


class PreparedStep:
    """lf_step_prepare / lf_step_run: one layer's decode step with its buffers,
    shape, plan and stream fixed once; ``run()`` then enqueues the step with
    no argument checks (see include/lf_decode.h). The per-step buffers (q,
    new_k, new_v, write_slot, out, next_slot) may each be CUDA tensors, pinned
    host tensors (read and written in place) or other host tensors (staged);
    the caches and the mask are CUDA tensors. The object keeps the tensors
    alive; write each token's inputs into the same tensors."""

    def __init__(self, q, k_cache, v_cache, mask, new_k, new_v, write_slot, out, next_slot, W,
                 scale, stream=None):
        lib = load_library()
        B, Hq, Hkv, d, S = _shapes(q, k_cache)
        bf, i32 = torch.bfloat16, torch.int32
        _need(k_cache, "k_cache", bf, (B, Hkv, S, d), True)
        _need(v_cache, "v_cache", bf, (B, Hkv, S, d), True)
        _need(mask, "mask", i32, (B, Hkv, S), True)
        for t, name, dt, shape in ((q, "q", bf, (B, Hq, d)), (new_k, "new_k", bf, (B, Hkv, d)),
                                   (new_v, "new_v", bf, (B, Hkv, d)),
                                   (write_slot, "write_slot", i32, (B, Hkv)),
                                   (out, "out", bf, (B, Hq, d)),
                                   (next_slot, "next_slot", i32, (B, Hkv))):
            _need(t, name, dt, shape, t.is_cuda if isinstance(t, torch.Tensor) else True)
        if stream is None:
            stream = torch.cuda.current_stream()
        self._keep = (q, k_cache, v_cache, mask, new_k, new_v, write_slot, out, next_slot, stream)
        self._lib = lib
        self._h = ctypes.c_void_p(0)
        _check(lib, lib.lf_step_prepare(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), mask.data_ptr(),
            new_k.data_ptr(), new_v.data_ptr(), write_slot.data_ptr(), out.data_ptr(),
            next_slot.data_ptr(), B, Hq, Hkv, d, S, int(W), float(scale),
            _stream_handle(stream), ctypes.byref(self._h)))
        self._run = lib.lf_step_run

    def run(self):
        """Enqueue one step on the prepare-time stream (asynchronous)."""
        st = self._run(self._h)
        if st:
            _check(self._lib, st)

    def errors(self, clear: bool = True) -> int:
        """OR of LF_DEVERR_* bits of this handle's runs (syncs its stream)."""
        flags = ctypes.c_uint32(0)
        _check(self._lib, self._lib.lf_step_errors(self._h, ctypes.byref(flags), int(clear)))
        return int(flags.value)

    def close(self):
        """Synchronise the stream and free the handle (idempotent)."""
        if self._h and self._h.value:
            h, self._h = self._h, ctypes.c_void_p(0)
            _check(self._lib, self._lib.lf_step_destroy(h))

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _Here:
    """The guard of a call on the current device: nothing to switch."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_HERE = _Here()
_gpus = 0  # visible GPUs, once known


def _on_device(device, *tensors):
    """The device guard of a call on `device`, where every tensor has to be."""
    global _gpus
    if _gpus == 0:
        _gpus = torch.cuda.device_count()
    if _gpus == 1:  # CUDA tensors cannot be anywhere else
        return _HERE
    index = device.index
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on {device} and {t.device}: all must be on one device")
    return _HERE if torch.cuda.current_device() == index else torch.cuda.device(device)


# The current stream's handle without a Stream object, where torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing",
                     torch.cuda.is_current_stream_capturing)


def _call_stream(stream, device):
    """_stream_handle for a call on `device`."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(device.index)
    return _stream_handle(stream)


# Workspaces of calls that bring none, per thread, device and stream: a
# thread's calls on a stream run one after the other. Calls that may outlive
# that order take their own from torch's allocator: captured ones (from the
# graph's pool) and those on a stream named by the caller.
_held = threading.local()


def _workspace(workspace, nbytes, device, stream):
    """The caller's workspace, or one of at least nbytes for this call."""
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
            raise TypeError("workspace: expected a uint8 torch.Tensor")
        if not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace: must be a contiguous tensor on {device}")
        return workspace
    if stream is None:
        if _raw_stream is None or _capturing():
            return torch.empty(nbytes, dtype=torch.uint8, device=device)
        key = (device.index, _raw_stream(device.index))
        held = _held.__dict__
        ws = held.get(key)
        if ws is None or ws.numel() < nbytes:
            held[key] = ws = torch.empty(nbytes + nbytes // 4, dtype=torch.uint8, device=device)
        return ws
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                  else torch.cuda.default_stream(device))
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_qkv(qkv, q_weight, k_weight, inv_freq, q_out, Hkv):
    T, Hq, d = _rope_shape(qkv, q_weight, k_weight, inv_freq, q_out)
    bf = torch.bfloat16
    _need(q_out, "q_out", bf, (T, Hq, d), True)
    if q_weight is not None:
        _need(q_weight, "q_weight", bf, (d,), True)
        _need(k_weight, "k_weight", bf, (d,), True)
    _need(inv_freq, "inv_freq", torch.float32, (inv_freq.numel(),), True)
    return T, Hq, d, 2 * inv_freq.numel(), _qkv_stride(qkv, T, Hq, Hkv, d)


def _rope_shape(qkv, q_weight, k_weight, inv_freq, q_out):
    if not isinstance(qkv, torch.Tensor) or not isinstance(q_out, torch.Tensor):
        raise TypeError("qkv and q_out: expected torch.Tensors")
    if q_out.dim() != 3 or qkv.dim() != 3:
        raise ValueError("qkv must be [T,Hq+2*Hkv,d] and q_out [T,Hq,d]")
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight must both be given or both be None")
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a [rot/2] tensor")
    return q_out.shape


def _qkv_stride(qkv, T, Hq, Hkv, d):
    """Elements between the rows of qkv, which may be strided."""
    if qkv.dtype != torch.bfloat16:
        raise TypeError(f"qkv: dtype {qkv.dtype}, expected {torch.bfloat16}")
    if tuple(qkv.shape) != (T, Hq + 2 * Hkv, d):
        raise ValueError(f"qkv: shape {tuple(qkv.shape)}, expected {(T, Hq + 2 * Hkv, d)}")
    if not qkv.is_cuda:
        raise ValueError("qkv: must be a CUDA tensor")
    stride, head, one = qkv.stride()
    if one != 1 or head != d:
        raise ValueError("qkv: a row's heads must be contiguous")
    if T == 1:
        stride = max(int(stride), (Hq + 2 * Hkv) * d)
        if stride % 8:
            stride = (Hq + 2 * Hkv) * d  # a single row has no stride to speak of
    return stride


def qk_norm_rope(qkv, q_weight, k_weight, inv_freq, positions, q_out, k_out, v_out, eps=1e-6,
                 interleaved=False, stream=None):
    """lf_qk_norm_rope: per-head norm (weights None: none) and rotation of the
    query and key heads of qkv [T,Hq+2*Hkv,d] (rows may be strided), values
    copied, into q_out [T,Hq,d] and k_out, v_out [T,Hkv,d]: decode_step's q,
    new_k and new_v for T = B. inv_freq [rot/2] fp32, positions [T] int32."""
    lib = load_library()
    if not isinstance(k_out, torch.Tensor) or k_out.dim() != 3:
        raise ValueError("k_out must be [T,Hkv,d]")
    Hkv = int(k_out.shape[1])
    T, Hq, d, rot, stride = _check_qkv(qkv, q_weight, k_weight, inv_freq, q_out, Hkv)
    bf = torch.bfloat16
    _need(k_out, "k_out", bf, (T, Hkv, d), True)
    _need(v_out, "v_out", bf, (T, Hkv, d), True)
    _need(positions, "positions", torch.int32, (T,), True)
    with _on_device(qkv.device, q_weight, k_weight, inv_freq, positions, q_out, k_out, v_out):
        _check(lib, lib.lf_qk_norm_rope(
            qkv.data_ptr(), stride, _ptr(q_weight), _ptr(k_weight), inv_freq.data_ptr(),
            positions.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), T, Hq, Hkv,
            d, rot, int(bool(interleaved)), float(eps), _call_stream(stream, qkv.device)))


def prefill_append(qkv, q_weight, k_weight, inv_freq, q_start, kv_len, q_out, k_cache, v_cache,
                   mask, eps=1e-6, interleaved=False, pos_offset=None, stream=None):
    """lf_prefill_append: qk_norm_rope of prompt tokens, their keys, values and
    ages straight into the caches. Rows q_start[b]..q_start[b+1] of qkv are
    the last tokens of sequence b's kv_len[b]."""
    lib = load_library()
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [B,Hkv,S,d]")
    B, Hkv, S, _ = k_cache.shape
    T, Hq, d, rot, stride = _check_qkv(qkv, q_weight, k_weight, inv_freq, q_out, Hkv)
    bf, i32 = torch.bfloat16, torch.int32
    _need(k_cache, "k_cache", bf, (B, Hkv, S, d), True)
    _need(v_cache, "v_cache", bf, (B, Hkv, S, d), True)
    _need(mask, "mask", i32, (B, Hkv, S), True)
    _need(q_start, "q_start", i32, (B + 1,), True)
    _need(kv_len, "kv_len", i32, (B,), True)
    if pos_offset is not None:
        _need(pos_offset, "pos_offset", i32, (B,), True)
    with _on_device(qkv.device, q_weight, k_weight, inv_freq, q_start, kv_len, pos_offset, q_out,
                    k_cache, v_cache, mask):
        _check(lib, lib.lf_prefill_append(
            qkv.data_ptr(), stride, _ptr(q_weight), _ptr(k_weight), inv_freq.data_ptr(),
            q_start.data_ptr(), kv_len.data_ptr(), _ptr(pos_offset), q_out.data_ptr(),
            k_cache.data_ptr(), v_cache.data_ptr(), mask.data_ptr(), T, B, Hq, Hkv, d, S, rot,
            int(bool(interleaved)), float(eps), _call_stream(stream, qkv.device)))


def _check_axes(positions, pair_axis, rot):
    """(axes, the pairs' axes as bytes)."""
    if not isinstance(positions, torch.Tensor) or positions.dim() != 2:
        raise ValueError("positions must be [axes,T]")
    if isinstance(pair_axis, torch.Tensor) and pair_axis.is_cuda:
        raise ValueError("pair_axis: expected rot/2 axes on the host")
    try:
        if not isinstance(pair_axis, bytes):
            # (Entry by entry: bytes() would take an array's memory as it lies.)
            pair_axis = pair_axis.tolist() if isinstance(pair_axis, torch.Tensor) else list(pair_axis)
        pairs = bytes(pair_axis)
    except (TypeError, ValueError) as e:
        raise ValueError(f"pair_axis: expected rot/2 axes, {e}") from None
    if len(pairs) != rot // 2:
        raise ValueError(f"pair_axis: {len(pairs)} entries, expected {rot // 2}")
    return positions.shape[0], pairs


def qk_norm_rope_axes(qkv, q_weight, k_weight, inv_freq, positions, pair_axis, q_out, k_out, v_out,
                      eps=1e-6, interleaved=False, stream=None):
    """lf_qk_norm_rope_axes: qk_norm_rope with a position on each of several axes,
    positions [axes,T] int32. pair_axis: the axis of each rotated pair, rot/2
    integers on the host (a list, bytes or CPU tensor)."""
    lib = _lib or load_library()
    if not isinstance(k_out, torch.Tensor) or k_out.dim() != 3:
        raise ValueError("k_out must be [T,Hkv,d]")
    Hkv = k_out.shape[1]
    T, Hq, d = _rope_shape(qkv, q_weight, k_weight, inv_freq, q_out)
    half = inv_freq.shape[0]
    axes, pairs = _check_axes(positions, pair_axis, 2 * half)
    bf = torch.bfloat16
    qo, ko, vo, pos, freq, wq, wk = _pointers(
        q_out, "q_out", bf, (T, Hq, d), k_out, "k_out", bf, (T, Hkv, d), v_out, "v_out", bf, (T, Hkv, d),
        positions, "positions", torch.int32, (axes, T), inv_freq, "inv_freq", torch.float32, (half,),
        q_weight, "q_weight", bf, (d,), k_weight, "k_weight", bf, (d,))
    stride = _qkv_stride(qkv, T, Hq, Hkv, d)
    device = qkv.device
    with _on_device(device, q_out):
        _check(lib, lib.lf_qk_norm_rope_axes(
            qkv.data_ptr(), stride, wq, wk, freq, pos, pairs, axes, qo, ko, vo, T, Hq, Hkv, d, 2 * half,
            int(bool(interleaved)), float(eps), _call_stream(stream, device)))


def prefill_append_axes(qkv, q_weight, k_weight, inv_freq, q_start, kv_len, positions, pair_axis,
                        q_out, k_cache, v_cache, mask, eps=1e-6, interleaved=False, stream=None):
    """lf_prefill_append_axes: prefill_append with the rotation's positions given per
    row and axis, positions [axes,T] int32 (slots still follow q_start and kv_len)."""
    lib = _lib or load_library()
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [B,Hkv,S,d]")
    B, Hkv, S, _ = k_cache.shape
    T, Hq, d = _rope_shape(qkv, q_weight, k_weight, inv_freq, q_out)
    half = inv_freq.shape[0]
    axes, pairs = _check_axes(positions, pair_axis, 2 * half)
    bf, i32 = torch.bfloat16, torch.int32
    qo, kc, vc, m, qs, kl, pos, freq, wq, wk = _pointers(
        q_out, "q_out", bf, (T, Hq, d), k_cache, "k_cache", bf, (B, Hkv, S, d),
        v_cache, "v_cache", bf, (B, Hkv, S, d), mask, "mask", i32, (B, Hkv, S),
        q_start, "q_start", i32, (B + 1,), kv_len, "kv_len", i32, (B,),
        positions, "positions", i32, (axes, T), inv_freq, "inv_freq", torch.float32, (half,),
        q_weight, "q_weight", bf, (d,), k_weight, "k_weight", bf, (d,))
    stride = _qkv_stride(qkv, T, Hq, Hkv, d)
    device = qkv.device
    with _on_device(device, q_out):
        _check(lib, lib.lf_prefill_append_axes(
            qkv.data_ptr(), stride, wq, wk, freq, qs, kl, pos, pairs, axes, qo, kc, vc, m, T, B, Hq,
            Hkv, d, S, 2 * half, int(bool(interleaved)), float(eps), _call_stream(stream, device)))


def window_attention_workspace(T, B, Hq, Hkv, d, S, window=0, sinks=0) -> int:
    """Workspace bytes of window_attention for these sizes on the current device."""
    lib = load_library()
    n = ctypes.c_size_t(0)
    _check(lib, lib.lf_window_attention_workspace(int(T), int(B), int(Hq), int(Hkv), int(d),
                                                  int(S), int(window), int(sinks),
                                                  ctypes.byref(n)))
    return int(n.value)


# The size is a function of the sizes and the device alone.
_window_bytes = functools.lru_cache(maxsize=1024)(
    lambda index, *sizes: window_attention_workspace(*sizes))


def window_attention(q, k_cache, v_cache, q_start, kv_len, out, window, sinks, scale,
                     workspace=None, stream=None):
    """lf_window_attention: packed rows q [T,Hq,d] over in-order caches
    [B,Hkv,S,d]; a token sees its last `window` keys (0: all) and the first
    `sinks`. workspace: uint8 of window_attention_workspace bytes (None: taken
    from torch's allocator; bring one to a capture that torch.cuda.graph does
    not make)."""
    lib = load_library()
    if not isinstance(q, torch.Tensor) or not isinstance(k_cache, torch.Tensor):
        raise TypeError("q and k_cache: expected torch.Tensors")
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [T,Hq,d] and k_cache [B,Hkv,S,d]")
    T, Hq, d = q.shape
    B, Hkv, S, _ = k_cache.shape
    bf, i32 = torch.bfloat16, torch.int32
    _need(q, "q", bf, (T, Hq, d), True)
    _need(k_cache, "k_cache", bf, (B, Hkv, S, d), True)
    _need(v_cache, "v_cache", bf, (B, Hkv, S, d), True)
    _need(q_start, "q_start", i32, (B + 1,), True)
    _need(kv_len, "kv_len", i32, (B,), True)
    _need(out, "out", bf, (T, Hq, d), True)
    with _on_device(q.device, k_cache, v_cache, q_start, kv_len, out):
        n = _window_bytes(q.device.index, T, B, Hq, Hkv, d, S, int(window), int(sinks))
        ws = _workspace(workspace, n, q.device, stream) if n or workspace is not None else None
        _check(lib, lib.lf_window_attention(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), q_start.data_ptr(),
            kv_len.data_ptr(), out.data_ptr(), T, B, Hq, Hkv, d, S, int(window), int(sinks),
            float(scale), _ptr(ws), 0 if ws is None else ws.numel(), _call_stream(stream, q.device)))


def decode_prefix_workspace(B, Hq, Hkv, d, S, N, P) -> int:
    """Workspace bytes of the *_prefix calls for these sizes on the current device."""
    lib = load_library()
    n = ctypes.c_size_t(0)
    _check(lib, lib.lf_decode_prefix_workspace(int(B), int(Hq), int(Hkv), int(d), int(S), int(N),
                                               int(P), ctypes.byref(n)))
    return int(n.value)


# The size is a function of the sizes, the device and one switch alone.
_prefix_bytes = functools.lru_cache(maxsize=1024)(
    lambda index, chunk_tiles, *sizes: decode_prefix_workspace(*sizes))


def _check_prefix(k_prefix, v_prefix, prefix_start, prefix_len, Hkv, d):
    if not isinstance(k_prefix, torch.Tensor) or k_prefix.dim() != 4:
        raise ValueError("k_prefix must be [N,Hkv,P,d]")
    N, P = int(k_prefix.shape[0]), int(k_prefix.shape[2])
    bf, i32 = torch.bfloat16, torch.int32
    _need(k_prefix, "k_prefix", bf, (N, Hkv, P, d), True)
    _need(v_prefix, "v_prefix", bf, (N, Hkv, P, d), True)
    _need(prefix_start, "prefix_start", i32, (N + 1,), True)
    _need(prefix_len, "prefix_len", i32, (N,), True)
    return N, P


def decode_attention_prefix(q, k_cache, v_cache, mask, new_k, new_v, write_slot, k_prefix,
                            v_prefix, prefix_start, prefix_len, out, scale, workspace=None,
                            stream=None):
    """lf_decode_attention_prefix: decode_attention whose sequences
    prefix_start[n]..prefix_start[n+1] also see the prefix_len[n] tokens of
    prefix n (k_prefix, v_prefix [N,Hkv,P,d]), in one softmax."""
    lib = load_library()
    B, Hq, Hkv, d, S = _shapes(q, k_cache)
    bf, i32 = torch.bfloat16, torch.int32
    _need(q, "q", bf, (B, Hq, d), True)
    _need(k_cache, "k_cache", bf, (B, Hkv, S, d), True)
    _need(v_cache, "v_cache", bf, (B, Hkv, S, d), True)
    _need(mask, "mask", i32, (B, Hkv, S), True)
    _need(new_k, "new_k", bf, (B, Hkv, d), True)
    _need(new_v, "new_v", bf, (B, Hkv, d), True)
    _need(write_slot, "write_slot", i32, (B, Hkv), True)
    _need(out, "out", bf, (B, Hq, d), True)
    N, P = _check_prefix(k_prefix, v_prefix, prefix_start, prefix_len, Hkv, d)
    with _on_device(q.device, k_cache, v_cache, mask, new_k, new_v, write_slot, out, k_prefix,
                    v_prefix, prefix_start, prefix_len):
        ws = _workspace(workspace, 0 if workspace is not None else
                        _prefix_bytes(q.device.index, os.environ.get("LF_CHUNK_TILES"), B, Hq, Hkv,
                                      d, S, N, P), q.device, stream)
        _check(lib, lib.lf_decode_attention_prefix(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), mask.data_ptr(),
            new_k.data_ptr(), new_v.data_ptr(), write_slot.data_ptr(), k_prefix.data_ptr(),
            v_prefix.data_ptr(), prefix_start.data_ptr(), prefix_len.data_ptr(), out.data_ptr(),
            B, Hq, Hkv, d, S, N, P, float(scale), ws.data_ptr(), ws.numel(),
            _call_stream(stream, q.device)))


def decode_step_prefix(q, k_cache, v_cache, mask, new_k, new_v, write_slot, k_prefix, v_prefix,
                       prefix_start, prefix_len, out, next_slots, W, scale, k=None, flags=0,
                       scores=None, workspace=None, stream=None):
    """lf_decode_step_prefix: decode_step_ex over shared prefixes and the
    sequences' own slots. next_slots [B,Hkv] (k None: the argmin) or
    [B,Hkv,k]; only own slots are scored, with weights normalised over both."""
    lib = load_library()
    B, Hq, Hkv, d, S = _check_step(q, k_cache, v_cache, mask, new_k, new_v, write_slot, out,
                                   next_slots, k=k)
    if scores is not None:
        _need(scores, "scores", torch.float32, (B, Hkv, S), True)
    N, P = _check_prefix(k_prefix, v_prefix, prefix_start, prefix_len, Hkv, d)
    with _on_device(q.device, k_cache, v_cache, mask, new_k, new_v, write_slot, out, next_slots,
                    scores, k_prefix, v_prefix, prefix_start, prefix_len):
        ws = _workspace(workspace, 0 if workspace is not None else
                        _prefix_bytes(q.device.index, os.environ.get("LF_CHUNK_TILES"), B, Hq, Hkv,
                                      d, S, N, P), q.device, stream)
        _check(lib, lib.lf_decode_step_prefix(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), mask.data_ptr(),
            new_k.data_ptr(), new_v.data_ptr(), write_slot.data_ptr(), k_prefix.data_ptr(),
            v_prefix.data_ptr(), prefix_start.data_ptr(), prefix_len.data_ptr(), out.data_ptr(),
            next_slots.data_ptr(), 1 if k is None else int(k), int(flags),
            None if scores is None else scores.data_ptr(), B, Hq, Hkv, d, S, N, P, int(W),
            float(scale), ws.data_ptr(), ws.numel(), _call_stream(stream, q.device)))


def decode_weights_workspace(B, Hq, Hkv, d, S, k=1) -> int:
    """Workspace bytes of decode_step_weights for these sizes on the current device."""
    lib = load_library()
    n = ctypes.c_size_t(0)
    _check(lib, lib.lf_decode_weights_workspace(int(B), int(Hq), int(Hkv), int(d), int(S), int(k),
                                                ctypes.byref(n)))
    return int(n.value)


# The size is a function of the sizes and the device, and of the plan's switches:
# a call that finds it too small asks again.
_weights_bytes = functools.lru_cache(maxsize=1024)(
    lambda index, *sizes: decode_weights_workspace(*sizes))


def decode_step_weights(q, k_cache, v_cache, mask, weights, new_k, new_v, write_slot, out,
                        next_slots, W, scale, decay=1.0, k=None, flags=0, workspace=None,
                        stream=None):
    """lf_decode_step_weights: the decode step that adds the token's attention weights
    to weights [B,Hkv,S] fp32 (decay * old + new) and returns the slots with the
    least. next_slots [B,Hkv] (k None: the argmin) or [B,Hkv,k]."""
    lib = _lib or load_library()
    B, Hq, Hkv, d, S = _shapes(q, k_cache)
    bf, i32 = torch.bfloat16, torch.int32
    topk = 1 if k is None else int(k)
    ptrs = _pointers(
        q, "q", bf, (B, Hq, d), k_cache, "k_cache", bf, (B, Hkv, S, d),
        v_cache, "v_cache", bf, (B, Hkv, S, d), mask, "mask", i32, (B, Hkv, S),
        weights, "weights", torch.float32, (B, Hkv, S), new_k, "new_k", bf, (B, Hkv, d),
        new_v, "new_v", bf, (B, Hkv, d), write_slot, "write_slot", i32, (B, Hkv),
        out, "out", bf, (B, Hq, d),
        next_slots, "next_slots", i32, (B, Hkv) if k is None else (B, Hkv, topk))
    device = q.device
    with _on_device(device, q):
        handle = _call_stream(stream, device)

        def call(ws):
            return lib.lf_decode_step_weights(*ptrs, topk, int(flags), B, Hq, Hkv, d, S, int(W),
                                              float(scale), float(decay), ws.data_ptr(), ws.numel(),
                                              handle)

        n = 0 if workspace is not None else _weights_bytes(device.index, B, Hq, Hkv, d, S, topk)
        ws = _workspace(workspace, n, device, stream)
        status = call(ws)
        if status == LF_ERR_INVALID_ARG and workspace is None:
            # (Nothing was enqueued.) The plan's switches may have changed.
            n = decode_weights_workspace(B, Hq, Hkv, d, S, topk)
            status = call(_workspace(None, n, device, stream) if n > ws.numel() else ws)
        _check(lib, status)


def prompt_weights_workspace(T, B, Hq, Hkv, d, S, rows=0) -> int:
    """Workspace bytes of prompt_weights for these sizes on the current device."""
    lib = load_library()
    n = ctypes.c_size_t(0)
    _check(lib, lib.lf_prompt_weights_workspace(int(T), int(B), int(Hq), int(Hkv), int(d), int(S),
                                                int(rows), ctypes.byref(n)))
    return int(n.value)


# The size is a function of the sizes and the device alone.
_prompt_bytes = functools.lru_cache(maxsize=1024)(
    lambda index, *sizes: prompt_weights_workspace(*sizes))


def prompt_weights(q, k_cache, q_start, kv_len, weights, scale, rows=0, workspace=None, stream=None):
    """lf_prompt_weights: the causal attention weights that the last `rows` rows (0:
    all) of each sequence give its keys, into weights [B,Hkv,S] fp32 (set for this
    call's tokens, added for earlier ones): decode_step_weights' start."""
    lib = _lib or load_library()
    if not isinstance(q, torch.Tensor) or not isinstance(k_cache, torch.Tensor):
        raise TypeError("q and k_cache: expected torch.Tensors")
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [T,Hq,d] and k_cache [B,Hkv,S,d]")
    T, Hq, d = q.shape
    B, Hkv, S, _ = k_cache.shape
    i32 = torch.int32
    ptrs = _pointers(
        q, "q", torch.bfloat16, (T, Hq, d), k_cache, "k_cache", torch.bfloat16, (B, Hkv, S, d),
        q_start, "q_start", i32, (B + 1,), kv_len, "kv_len", i32, (B,),
        weights, "weights", torch.float32, (B, Hkv, S))
    device = q.device
    with _on_device(device, q):
        n = 0 if workspace is not None else _prompt_bytes(device.index, T, B, Hq, Hkv, d, S, int(rows))
        ws = _workspace(workspace, n, device, stream)
        _check(lib, lib.lf_prompt_weights(*ptrs, T, B, Hq, Hkv, d, S, int(rows), float(scale),
                                          ws.data_ptr(), ws.numel(), _call_stream(stream, device)))


def _kv4_shape(k4):
    """(B, Hkv, S, d) of a 4-bit cache's keys."""
    if not isinstance(k4, torch.Tensor) or k4.dim() != 4:
        raise ValueError("k4 must be [B,Hkv,S,d/2]")
    B, Hkv, S, half = k4.shape
    return B, Hkv, S, 2 * half


def _kv4_slots(k4, k_scale, v4, v_scale, kv_from, kv_len, k_cache, v_cache, mask):
    """The sizes and pointers of a call that packs or unpacks (mask None)."""
    B, Hkv, S, d = _kv4_shape(k4)
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [B,Hkv,P,d]")
    P = k_cache.shape[2]
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    return (B, Hkv, d, P, S), _pointers(
        k4, "k4", u8, (B, Hkv, S, d // 2), k_scale, "k_scale", bf, (B, Hkv, S, d // 32),
        v4, "v4", u8, (B, Hkv, S, d // 2), v_scale, "v_scale", bf, (B, Hkv, S, d // 32),
        kv_from, "kv_from", i32, (B,), kv_len, "kv_len", i32, (B,),
        k_cache, "k_cache", bf, (B, Hkv, P, d), v_cache, "v_cache", bf, (B, Hkv, P, d),
        mask, "mask", i32, (B, Hkv, S))


def kv4_pack(k_cache, v_cache, kv_from, kv_len, k4, k_scale, v4, v_scale, mask, stream=None):
    """lf_kv4_pack: slots kv_from[b]..kv_len[b] (kv_from None: from 0) of bf16 caches
    [B,Hkv,P,d] into a 4-bit cache: k4, v4 uint8 [B,Hkv,S,d/2], k_scale, v_scale
    bf16 [B,Hkv,S,d/32]; mask [B,Hkv,S] gets the ages of an in-order cache."""
    lib = _lib or load_library()
    if kv_len is None or mask is None:
        raise TypeError("kv_len and mask: expected torch.Tensors")
    sizes, (c, cs, w, wsc, first, last, kc, vc, m) = _kv4_slots(
        k4, k_scale, v4, v_scale, kv_from, kv_len, k_cache, v_cache, mask)
    device = k4.device
    with _on_device(device, k4):
        _check(lib, lib.lf_kv4_pack(kc, vc, first, last, c, cs, w, wsc, m, *sizes,
                                    _call_stream(stream, device)))


def kv4_unpack(k4, k_scale, v4, v_scale, kv_from, kv_len, k_cache, v_cache, stream=None):
    """lf_kv4_unpack: the values of slots kv_from[b]..kv_len[b] of a 4-bit cache back
    into bf16 caches [B,Hkv,P,d]."""
    lib = _lib or load_library()
    if kv_len is None:
        raise TypeError("kv_len: expected a torch.Tensor")
    sizes, (c, cs, w, wsc, first, last, kc, vc, _) = _kv4_slots(
        k4, k_scale, v4, v_scale, kv_from, kv_len, k_cache, v_cache, None)
    device = k4.device
    with _on_device(device, k4):
        _check(lib, lib.lf_kv4_unpack(c, cs, w, wsc, first, last, kc, vc, *sizes,
                                      _call_stream(stream, device)))


def decode_kv4_workspace(B, Hq, Hkv, d, S) -> int:
    """Workspace bytes of decode_attention_kv4 for these sizes on the current device."""
    lib = load_library()
    n = ctypes.c_size_t(0)
    _check(lib, lib.lf_decode_kv4_workspace(int(B), int(Hq), int(Hkv), int(d), int(S), ctypes.byref(n)))
    return int(n.value)


# The size is a function of the sizes and the device alone.
_kv4_bytes = functools.lru_cache(maxsize=1024)(lambda index, *sizes: decode_kv4_workspace(*sizes))


def decode_attention_kv4(q, k4, k_scale, v4, v_scale, mask, new_k, new_v, write_slot, out, scale,
                         workspace=None, stream=None):
    """lf_decode_attention_kv4: decode_attention over a 4-bit cache (the token's row
    is put into 4 bits in write_slot and attended as the values it then stands for)."""
    lib = _lib or load_library()
    B, Hkv, S, d = _kv4_shape(k4)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [B,Hq,d]")
    Hq = q.shape[1]
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    ptrs = _pointers(
        q, "q", bf, (B, Hq, d), k4, "k4", u8, (B, Hkv, S, d // 2),
        k_scale, "k_scale", bf, (B, Hkv, S, d // 32), v4, "v4", u8, (B, Hkv, S, d // 2),
        v_scale, "v_scale", bf, (B, Hkv, S, d // 32), mask, "mask", i32, (B, Hkv, S),
        new_k, "new_k", bf, (B, Hkv, d), new_v, "new_v", bf, (B, Hkv, d),
        write_slot, "write_slot", i32, (B, Hkv), out, "out", bf, (B, Hq, d))
    device = q.device
    with _on_device(device, q):
        n = _kv4_bytes(device.index, B, Hq, Hkv, d, S)
        ws = _workspace(workspace, n, device, stream) if n or workspace is not None else None
        _check(lib, lib.lf_decode_attention_kv4(
            *ptrs, B, Hq, Hkv, d, S, float(scale), _ptr(ws), 0 if ws is None else ws.numel(),
            _call_stream(stream, device)))


def step_plan(B: int, Hq: int, Hkv: int, d: int, S: int, topk: int = 1) -> dict:
    """The launch plan a step of this shape takes on the current device."""
    lib = load_library()
    plan = (ctypes.c_int32 * 6)()
    _check(lib, lib.lf_step_plan(int(B), int(Hq), int(Hkv), int(d), int(S), int(topk), plan))
    return {"nchunk": plan[0], "chunk_tiles": plan[1], "stages": plan[2],
            "cluster": bool(plan[3]), "split": bool(plan[4]), "cluster_fit": plan[5]}


def device_errors(stream=None, clear: bool = True) -> int:
    """OR of LF_DEVERR_* bits raised on `stream` since the last clear (syncs the stream)."""
    lib = load_library()
    flags = ctypes.c_uint32(0)
    _check(lib, lib.lf_device_errors(_stream_handle(stream), ctypes.byref(flags), int(clear)))
    return int(flags.value)


def profile_enable(on: bool = True):
    lib = load_library()
    _check(lib, lib.lf_profile_enable(int(on)))


def profile_collect(kernel_id: int):
    """(total event milliseconds, launches) for one kernel id since the last collect."""
    lib = load_library()
    ms = ctypes.c_double(0)
    n = ctypes.c_int64(0)
    _check(lib, lib.lf_profile_collect(int(kernel_id), ctypes.byref(ms), ctypes.byref(n)))
    return float(ms.value), int(n.value)


def release_workspace():
    """Free the library's scratch, and this thread's workspaces."""
    lib = load_library()
    _held.__dict__.clear()
    _check(lib, lib.lf_release_workspace())


def status_string(status: int) -> str:
    return load_library().lf_status_string(int(status)).decode()


def version() -> int:
    return int(load_library().lf_version())
