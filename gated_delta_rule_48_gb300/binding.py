"""ctypes binding of ``libkda.so`` (the C ABI in ``include/kda.h``).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  torch supplies device memory and the current stream.  There is no
fallback: if the library is missing or no GPU is present, calls raise.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import threading
import warnings

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_CSRC = os.path.join(_PKG, "csrc")
_INCLUDE = os.path.join(os.path.dirname(_PKG), "include")
_BUILD = os.path.join(_PKG, "_build")
_LIB = os.path.join(_BUILD, "libkda.so")
# the bounds-checked build (-DKDA_BOUNDS_CHECK), objects and library apart
_BUILD_CHECKED = os.path.join(_BUILD, "checked")
_LIB_CHECKED = os.path.join(_BUILD_CHECKED, "libkda.so")
# the module that takes torch tensors to the library's operators (csrc/kda_torch.cpp), for the
# torch at hand
_EXT = os.path.join(_BUILD, f"torch-{torch.__version__}", "kda_torch.so")
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]

_lock = threading.Lock()
_libs = {}          # False: the normal library, True: the bounds-checked one
_checked = False    # which one load() returns
_extension = None   # the module of csrc/kda_torch.cpp
_selected = None    # the same, once its calls go to the library that load() returns

STATUS = {0: "KDA_OK", 1: "KDA_ERR_INVALID_ARGUMENT", 2: "KDA_ERR_UNSUPPORTED",
          3: "KDA_ERR_CUDA", 4: "KDA_ERR_OUT_OF_MEMORY", 5: "KDA_ERR_DEVICE_INPUT"}


class KdaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


def library_path() -> str:
    return _LIB_CHECKED if _checked else _LIB


def use_checked(checked: bool) -> None:
    """Route every call of this module to the bounds-checked library (True)
    or to the normal one (False, the default).  Both may be loaded at once;
    each keeps its own device state."""
    global _checked, _selected
    _checked = bool(checked)
    _selected = None


def _sources():
    return sorted(os.path.join(_CSRC, f) for f in os.listdir(_CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(_CSRC, f) for f in os.listdir(_CSRC) if f.endswith((".h", ".cuh"))]
    return hs + [os.path.join(_INCLUDE, "kda.h")]


def _build_extension(force: bool = False):
    """(command, process) of the compilation of ``csrc/kda_torch.cpp``, or None when it is up to
    date.  ``_EXT`` is in place once :func:`build` has waited for it."""
    src = os.path.join(_CSRC, "kda_torch.cpp")
    newest = max(os.path.getmtime(p) for p in (src, os.path.join(_INCLUDE, "kda.h")))
    if not force and os.path.exists(_EXT) and os.path.getmtime(_EXT) >= newest:
        return None
    os.makedirs(os.path.dirname(_EXT), exist_ok=True)
    root = os.path.dirname(torch.__file__)
    nvcc = shutil.which("nvcc")
    cuda = os.path.dirname(os.path.dirname(nvcc)) if nvcc else "/usr/local/cuda"
    lib = os.path.join(root, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
           "-I", _INCLUDE, src, "-o", _EXT + f".tmp{os.getpid()}", "-L", lib, "-ltorch",
           "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}", "-ldl"]
    try:
        return cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except OSError as e:  # no such compiler
        return cmd, e


def _finish_extension(ext, verbose: bool = False) -> str:
    """Wait for what :func:`_build_extension` started.  Returns why it failed, or "" with
    ``_EXT`` in place; after a failure there is no (older) ``_EXT``."""
    if ext is None:
        return ""
    cmd, p = ext
    if isinstance(p, OSError):
        why = str(p)
    else:
        why = p.communicate()[0].decode(errors="replace")
        if verbose:
            print(why)
        if p.returncode == 0:
            os.replace(_EXT + f".tmp{os.getpid()}", _EXT)
            return ""
    if os.path.exists(_EXT):
        os.unlink(_EXT)
    return f"compilation failed:\n{' '.join(cmd)}\n{why}"


def _finish(procs, verbose):
    """Wait for the library's compilations; raise if one failed."""
    failed = []
    for cmd, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode:
            print(out.decode(errors="replace"))
        if p.returncode:
            failed.append(" ".join(cmd))
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(failed))


def _warn(failure: str):
    if failure:
        warnings.warn(f"the operators' Python calls are not available: {failure}", RuntimeWarning,
                      stacklevel=3)


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    """Compile every ``csrc/*.cu`` for sm_103a and link ``_build/libkda.so``
    (with ``checked``: ``_build/checked/libkda.so``, every kernel compiled with
    -DKDA_BOUNDS_CHECK).

    Translation units compile in parallel; nvcc cross-compiles, so no GPU is
    needed.  Rebuilds only when a source or header is newer than the library.

    The module that takes torch tensors to the operators is compiled beside it.
    The library does not need it (nor torch's and Python's headers): where it
    cannot be compiled that is a warning here, and an error of the operators'
    Python calls.
    """
    bdir, lib_path = (_BUILD_CHECKED, _LIB_CHECKED) if checked else (_BUILD, _LIB)
    os.makedirs(bdir, exist_ok=True)
    ext = _build_extension(force)
    srcs = _sources()
    newest = max(os.path.getmtime(p) for p in srcs + _headers())
    if not force and os.path.exists(lib_path) and os.path.getmtime(lib_path) >= newest:
        _warn(_finish_extension(ext, verbose))
        return lib_path
    common = ["nvcc", *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-I", _INCLUDE, "-I", _CSRC, "--expt-relaxed-constexpr"]
    if checked:
        common.append("-DKDA_BOUNDS_CHECK")
    objs, procs = [], []
    for src in srcs:
        obj = os.path.join(bdir, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = common + ["-c", src, "-o", obj]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                             stderr=subprocess.STDOUT)))
    failure = _finish_extension(ext, verbose)
    _finish(procs, verbose)
    tmp = lib_path + f".tmp{os.getpid()}"
    subprocess.check_call(["nvcc", *ARCH_FLAGS, "-shared", "-o", tmp, *objs])
    os.replace(tmp, lib_path)
    _warn(failure)  # (with the library in place, should warnings be errors)
    return lib_path


class KdaTensor(ctypes.Structure):
    """``kda_tensor`` of include/kda.h."""
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class KdaKv4Cache(ctypes.Structure):
    """``kda_kv4_cache`` of include/kda.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales")] + [
        (n, ctypes.c_int32) for n in ("n_pages", "page_size", "n_kv_heads", "d")]


KDA_DTYPE = {torch.bfloat16: 0, torch.float32: 1, torch.int32: 2, torch.float8_e4m3fn: 3}


def describe(t):
    """A kda_tensor for a torch tensor (None for None): pointer, dtype,
    shape and strides exactly as torch holds them, unchecked."""
    if t is None:
        return None
    d = KdaTensor()
    d.data = t.data_ptr()
    d.dtype = KDA_DTYPE.get(t.dtype, 99)
    d.ndim = t.dim()
    for i in range(t.dim()):
        d.shape[i] = t.shape[i]
        d.stride[i] = t.stride(i)
    return d


class _KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double)]


def load():
    """Load (building first if needed) the library; returns the ctypes handle."""
    lib = _libs.get(_checked)
    if lib is not None:
        return lib
    with _lock:
        if _checked not in _libs:
            path = library_path()
            if not os.path.exists(path):
                path = build(checked=_checked)
            lib = ctypes.CDLL(path)
            vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
            lib.kda_chunk_fwd.restype = ctypes.c_int
            lib.kda_chunk_fwd.argtypes = [vp] * 9 + [i64, i32, i32, i32, i32, vp]
            lib.kda_chunk_fwd_split.restype = ctypes.c_int
            lib.kda_chunk_fwd_split.argtypes = [vp] * 9 + [i64, i32, i32, i32, i32, i64, vp]
            lib.kda_chunk_fwd_noalloc.restype = ctypes.c_int
            lib.kda_chunk_fwd_noalloc.argtypes = [vp] * 9 + [i64, i32, i32, i32, i32, vp]
            lib.kda_decode_step.restype = ctypes.c_int
            lib.kda_decode_step.argtypes = [vp] * 7 + [i32, i32, i32, i32, vp]
            lib.kda_chunk_fwd_fused.restype = ctypes.c_int
            lib.kda_chunk_fwd_fused.argtypes = [vp] * 9 + [i64, i32, i32, i32, i32, vp]
            lib.kda_decode_step_fused.restype = ctypes.c_int
            lib.kda_decode_step_fused.argtypes = [vp] * 7 + [i32, i32, i32, i32, vp]
            lib.kda_chunk_fwd_checkpoints.restype = ctypes.c_int
            lib.kda_chunk_fwd_checkpoints.argtypes = ([vp] * 9 + [i64, i32, i32, i32, i32, i64, vp, i64, vp])
            lib.kda_chunk_fwd_host.restype = ctypes.c_int
            lib.kda_chunk_fwd_host.argtypes = [vp] * 8 + [i64, i32, i32, i32, i32, i64, vp]
            lib.kda_decode_tokens_fused.restype = ctypes.c_int
            lib.kda_decode_tokens_fused.argtypes = [vp] * 8 + [i32, i32, i32, i32, i32, vp]
            lib.kda_decode_tokens.restype = ctypes.c_int
            lib.kda_decode_tokens.argtypes = [vp] * 8 + [i32, i32, i32, i32, i32, vp]
            lib.kda_get_device_error.restype = ctypes.c_int
            lib.kda_get_device_error.argtypes = [vp]
            lib.kda_status_string.restype = ctypes.c_char_p
            lib.kda_status_string.argtypes = [ctypes.c_int]
            lib.kda_last_error_message.restype = ctypes.c_char_p
            lib.kda_last_error_message.argtypes = []
            lib.kda_abi_version.restype = ctypes.c_int
            tp = ctypes.POINTER(KdaTensor)
            lib.kda_chunk_fwd_t.restype = ctypes.c_int
            lib.kda_chunk_fwd_t.argtypes = [tp] * 9 + [vp]
            lib.kda_decode_step_t.restype = ctypes.c_int
            lib.kda_decode_step_t.argtypes = [tp] * 7 + [vp]
            lib.kda_debug_chunk_dump.restype = ctypes.c_int
            lib.kda_debug_chunk_dump.argtypes = [vp] * 9 + [i64, i32, i32, i32, i32, i32, i32, i64,
                                                         vp, vp]
            lib.kda_workspace_pool_bytes.restype = ctypes.c_int64
            lib.kda_workspace_pool_bytes.argtypes = []
            lib.kda_auto_segment_tokens.restype = ctypes.c_int64
            lib.kda_auto_segment_tokens.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                                    ctypes.c_int32, ctypes.c_int32]
            lib.kda_selftest_bounded_wait.restype = ctypes.c_int
            lib.kda_selftest_bounded_wait.argtypes = [ctypes.c_uint32, vp]
            lib.kda_selftest_bounds_check.restype = ctypes.c_int
            lib.kda_selftest_bounds_check.argtypes = [vp]
            lib.kda_bounds_checked.restype = ctypes.c_int
            lib.kda_bounds_checked.argtypes = []
            f32, i = ctypes.c_float, ctypes.c_int
            lib.kda_add_rms_norm.restype = i
            lib.kda_add_rms_norm.argtypes = [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, i64, i64,
                                             i32, f32, i, i, i, vp]
            lib.kda_short_conv_fwd.restype = i
            lib.kda_short_conv_fwd.argtypes = [vp, i64, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32,
                                               i32, i32, i, i, vp]
            lib.kda_short_conv_step.restype = i
            lib.kda_short_conv_step.argtypes = [vp, i64, vp, vp, vp, vp, i64, i32, i32, i32, i32, i,
                                                i, vp]
            lib.kda_ssm_scan_fwd.restype = i
            lib.kda_ssm_scan_fwd.argtypes = [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, i64, vp,
                                             vp, vp, vp, i64, vp, i64, i32, i32, i32, i32, i32, i,
                                             vp]
            lib.kda_ssm_scan_step.restype = i
            lib.kda_ssm_scan_step.argtypes = [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, i64,
                                              vp, vp, vp, i64, i32, i32, i32, i32, i32, i, vp]
            lib.kda_matmul_fp8.restype = i
            lib.kda_matmul_fp8.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32, i32,
                                           i32, i, vp]
            cp = ctypes.POINTER(KdaKv4Cache)
            lib.kda_attention_fwd.restype = i
            lib.kda_attention_fwd.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, i64,
                                              i32, i32, i32, i32, f32, i32, vp]
            for name in ("kda_kv4_write", "kda_kv4_read"):
                getattr(lib, name).restype = i
                getattr(lib, name).argtypes = [vp, i64, vp, i64, cp, vp, i64, i32, vp, vp, i64, i32, vp]
            lib.kda_kv4_attention.restype = i
            lib.kda_kv4_attention.argtypes = [vp, i64, cp, vp, i64, i32, vp, vp, i64, vp, i32, i32, i32,
                                              f32, vp]
            lib.kda_profile_enable.restype = None
            lib.kda_profile_enable.argtypes = [ctypes.c_int]
            lib.kda_profile_read.restype = ctypes.c_int
            lib.kda_profile_read.argtypes = [ctypes.POINTER(_KernelTime), ctypes.c_int]
            _libs[_checked] = lib
    return _libs[_checked]


def _check(status: int):
    if status != 0:
        msg = load().kda_last_error_message().decode(errors="replace")
        raise KdaError(status, msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _require(t, dtype, name):
    if t is None:
        return
    if not t.is_cuda:
        raise KdaError(1, f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise KdaError(1, f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise KdaError(1, f"{name} must be contiguous")


def kda_chunk_fwd(q, k, v, log_alpha, beta, S0=None, cu_seqlens=None, out=None,
                  S_final=None, *, n_seqs=None, segment_tokens=0, want_state=True,
                  stream=None, _fused=False):
    """Prefill.  Tensors in the packed layout of ``include/kda.h``.

    q, k: bf16 [T, H, dk] (or [B, T_b, H, dk], a uniform batch); v bf16;
    log_alpha f32; beta f32 [T, H]; S0 f32 [N, H, dk, dv] or None;
    cu_seqlens int32 [N+1] (CUDA) or None.  Returns (out, S_final).
    """
    if q.dim() == 4:  # uniform batch [B, T_b, H, d]
        B = q.shape[0]
        q, k, v = (x.reshape(-1, *x.shape[2:]) for x in (q, k, v))
        log_alpha = log_alpha.reshape(-1, *log_alpha.shape[2:])
        beta = beta.reshape(-1, beta.shape[-1])
        if n_seqs is None:
            n_seqs = B
    T, H, dk = q.shape
    dv = v.shape[-1]
    if cu_seqlens is not None:
        n_seqs = cu_seqlens.shape[0] - 1
    elif n_seqs is None:
        n_seqs = 1
    la_dt, la_name = (torch.bfloat16, "gate") if _fused else (torch.float32, "log_alpha")
    for t, dt, name in ((q, torch.bfloat16, "q"), (k, torch.bfloat16, "k"),
                        (v, torch.bfloat16, "v"), (log_alpha, la_dt, la_name),
                        (beta, torch.float32, "beta"), (S0, torch.float32, "S0"),
                        (cu_seqlens, torch.int32, "cu_seqlens")):
        _require(t, dt, name)
    if out is None:
        out = torch.empty((T, H, dv), dtype=torch.bfloat16, device=q.device)
    if S_final is None and want_state:
        S_final = torch.empty((n_seqs, H, dk, dv), dtype=torch.float32, device=q.device)
    _require(out, torch.bfloat16, "out")
    _require(S_final, torch.float32, "S_final")
    lib = load()
    args = [_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0),
            _ptr(cu_seqlens), _ptr(out), _ptr(S_final), T, n_seqs, H, dk, dv]
    if _fused:
        if segment_tokens:
            raise ValueError("the fused entry point chooses its own segments")
        _check(lib.kda_chunk_fwd_fused(*args, _stream(stream)))
    elif segment_tokens:
        _check(lib.kda_chunk_fwd_split(*args, int(segment_tokens), _stream(stream)))
    else:
        _check(lib.kda_chunk_fwd(*args, _stream(stream)))
    return out, S_final


def kda_chunk_fwd_fused(q_raw, k_raw, v, gate, beta, S0=None, cu_seqlens=None, out=None,
                        S_final=None, *, n_seqs=None, want_state=True, stream=None):
    """Prefill with the input preparation on load: q_raw, k_raw bf16 unnormalised,
    gate bf16 logits [T, H, dk] in place of log_alpha (log alpha = -5 sigmoid(gate)).
    Otherwise as :func:`kda_chunk_fwd`."""
    return kda_chunk_fwd(q_raw, k_raw, v, gate, beta, S0, cu_seqlens, out, S_final,
                         n_seqs=n_seqs, want_state=want_state, stream=stream, _fused=True)


def kda_decode_step(q, k, v, log_alpha, beta, S_inout, out=None, *, stream=None):
    """One decode step; ``S_inout`` [N, H, dk, dv] f32 is updated in place.

    q, k: bf16 [N, H, dk]; v bf16 [N, H, dv]; log_alpha f32 [N, H, dk];
    beta f32 [N, H].  Returns out bf16 [N, H, dv].
    """
    N, H, dk = q.shape
    dv = v.shape[-1]
    for t, dt, name in ((q, torch.bfloat16, "q"), (k, torch.bfloat16, "k"),
                        (v, torch.bfloat16, "v"), (log_alpha, torch.float32, "log_alpha"),
                        (beta, torch.float32, "beta"), (S_inout, torch.float32, "S_inout")):
        _require(t, dt, name)
    if out is None:
        out = torch.empty((N, H, dv), dtype=torch.bfloat16, device=q.device)
    _require(out, torch.bfloat16, "out")
    _check(load().kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                  _ptr(S_inout), _ptr(out), N, H, dk, dv, _stream(stream)))
    return out


def kda_decode_step_fused(q_raw, k_raw, v, gate, beta, S_inout, out=None, *, stream=None):
    """Decode step with the input preparation on load (see :func:`kda_chunk_fwd_fused`)."""
    N, H, dk = q_raw.shape
    dv = v.shape[-1]
    for t, dt, name in ((q_raw, torch.bfloat16, "q_raw"), (k_raw, torch.bfloat16, "k_raw"),
                        (v, torch.bfloat16, "v"), (gate, torch.bfloat16, "gate"),
                        (beta, torch.float32, "beta"), (S_inout, torch.float32, "S_inout")):
        _require(t, dt, name)
    if out is None:
        out = torch.empty((N, H, dv), dtype=torch.bfloat16, device=q_raw.device)
    _require(out, torch.bfloat16, "out")
    _check(load().kda_decode_step_fused(_ptr(q_raw), _ptr(k_raw), _ptr(v), _ptr(gate),
                                        _ptr(beta), _ptr(S_inout), _ptr(out), N, H, dk, dv,
                                        _stream(stream)))
    return out


def _dref(d):
    return None if d is None else ctypes.byref(d)


def kda_chunk_fwd_t(q, k, v, log_alpha, beta, S0=None, cu_seqlens=None, out=None, S_final=None,
                    *, stream=None):
    """The descriptor form of the prefill: tensors go to the library with their
    dtype, shape and strides, and the library checks them.  ``out`` and
    ``S_final`` must be given (None skips S_final)."""
    descs = [describe(t) for t in (q, k, v, log_alpha, beta, S0, cu_seqlens, out, S_final)]
    _check(load().kda_chunk_fwd_t(*[_dref(d) for d in descs], _stream(stream)))
    return out, S_final


def kda_decode_step_t(q, k, v, log_alpha, beta, S_inout, out, *, stream=None):
    """The descriptor form of the decode step (see :func:`kda_chunk_fwd_t`)."""
    descs = [describe(t) for t in (q, k, v, log_alpha, beta, S_inout, out)]
    _check(load().kda_decode_step_t(*[_dref(d) for d in descs], _stream(stream)))
    return out


DUMP_LAYOUT = {"g": (0, (64, 128)), "A_kk": (8192, (64, 64)), "A_qk": (12288, (64, 64)),
               "T": (16384, (64, 64)), "U": (20480, (64, 128)), "S": (28672, (128, 128))}
DUMP_FLOATS = 45056


def kda_debug_chunk_dump(q, k, v, log_alpha, beta, S0=None, cu_seqlens=None, *, n_seqs=None,
                         seq, head, chunk, stream=None):
    """kda_chunk_fwd (never split) plus the intermediates of one chunk.

    Returns (out, S_final, {name: tensor}) with the names of DUMP_LAYOUT."""
    T, H, dk = q.shape
    dv = v.shape[-1]
    if cu_seqlens is not None:
        n_seqs = cu_seqlens.shape[0] - 1
    elif n_seqs is None:
        n_seqs = 1
    for t, dt, name in ((q, torch.bfloat16, "q"), (k, torch.bfloat16, "k"),
                        (v, torch.bfloat16, "v"), (log_alpha, torch.float32, "log_alpha"),
                        (beta, torch.float32, "beta"), (S0, torch.float32, "S0"),
                        (cu_seqlens, torch.int32, "cu_seqlens")):
        _require(t, dt, name)
    out = torch.empty((T, H, dv), dtype=torch.bfloat16, device=q.device)
    S_final = torch.empty((n_seqs, H, dk, dv), dtype=torch.float32, device=q.device)
    dump = torch.zeros(DUMP_FLOATS, dtype=torch.float32, device=q.device)
    _check(load().kda_debug_chunk_dump(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                       _ptr(S0), _ptr(cu_seqlens), _ptr(out), _ptr(S_final), T,
                                       n_seqs, H, dk, dv, int(seq), int(head), int(chunk),
                                       _ptr(dump), _stream(stream)))
    parts = {name: dump[off:off + int(np.prod(shape))].view(*shape)
             for name, (off, shape) in DUMP_LAYOUT.items()}
    return out, S_final, parts


def kda_auto_segment_tokens(total_tokens, n_seqs, n_heads, sm_count, uniform) -> int:
    """The segment length the automatic split picks (-1: no split); host only.
    ``uniform``: the batch has cu_seqlens None (sequences of equal length)."""
    return int(load().kda_auto_segment_tokens(total_tokens, n_seqs, n_heads, sm_count,
                                              1 if uniform else 0))


def kda_workspace_pool_bytes() -> int:
    """Bytes reserved by the library's workspace pool on the current device,
    or -1 when the library has created no pool there."""
    return int(load().kda_workspace_pool_bytes())


def kda_get_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status."""
    return load().kda_get_device_error(_stream(stream))


def kda_bounds_checked() -> bool:
    """Whether the loaded library is the bounds-checked build."""
    return bool(load().kda_bounds_checked())


def kda_selftest_bounds_check(*, stream=None):
    """One out-of-range guard, no memory access (see include/kda.h)."""
    _check(load().kda_selftest_bounds_check(_stream(stream)))


def kda_selftest_bounded_wait(polls: int = 1000, *, stream=None):
    """One bounded wait on an mbarrier nothing arrives on (see include/kda.h);
    the next kda_get_device_error() reports the timeout."""
    _check(load().kda_selftest_bounded_wait(int(polls), _stream(stream)))


def profile_enable(on: bool = True):
    load().kda_profile_enable(1 if on else 0)


def profile_read():
    """{kernel name: (launches, total ms)} since the last read."""
    buf = (_KernelTime * 32)()
    n = load().kda_profile_read(buf, 32)
    return {buf[i].name.decode(): (int(buf[i].launches), float(buf[i].total_ms))
            for i in range(n)}


def kda_decode_tokens(q, k, v, log_alpha, beta, S_inout, commit=None, out=None, *, stream=None):
    """K tokens per sequence from the state ``S_inout`` [N, H, dk, dv] f32.

    q, k: bf16 [N, K, H, dk]; v bf16 [N, K, H, dv]; log_alpha f32 [N, K, H, dk];
    beta f32 [N, K, H]; commit: int32 [N] (CUDA) or None (commit all K).
    Returns out bf16 [N, K, H, dv]; ``S_inout`` holds the state after the
    committed tokens of each sequence.
    """
    N, K, H, dk = q.shape
    dv = v.shape[-1]
    for t, dt, name in ((q, torch.bfloat16, "q"), (k, torch.bfloat16, "k"),
                        (v, torch.bfloat16, "v"), (log_alpha, torch.float32, "log_alpha"),
                        (beta, torch.float32, "beta"), (S_inout, torch.float32, "S_inout"),
                        (commit, torch.int32, "commit")):
        _require(t, dt, name)
    if out is None:
        out = torch.empty((N, K, H, dv), dtype=torch.bfloat16, device=q.device)
    _require(out, torch.bfloat16, "out")
    _check(load().kda_decode_tokens(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                    _ptr(S_inout), _ptr(out), _ptr(commit), N, K, H, dk, dv,
                                    _stream(stream)))
    return out


def kda_chunk_fwd_checkpoints(q, k, v, log_alpha, beta, S0=None, cu_seqlens=None, *, interval,
                              max_checkpoints, n_seqs=None, stream=None):
    """Prefill that also returns the state after every ``interval`` tokens of each
    sequence (see include/kda.h).  Returns (out, S_final, checkpoints), checkpoints
    f32 [max_checkpoints, H, dk, dv] packed sequence by sequence."""
    T, H, dk = q.shape
    dv = v.shape[-1]
    if cu_seqlens is not None:
        n_seqs = cu_seqlens.shape[0] - 1
    elif n_seqs is None:
        n_seqs = 1
    for t, dt, name in ((q, torch.bfloat16, "q"), (k, torch.bfloat16, "k"),
                        (v, torch.bfloat16, "v"), (log_alpha, torch.float32, "log_alpha"),
                        (beta, torch.float32, "beta"), (S0, torch.float32, "S0"),
                        (cu_seqlens, torch.int32, "cu_seqlens")):
        _require(t, dt, name)
    out = torch.empty((T, H, dv), dtype=torch.bfloat16, device=q.device)
    S_final = torch.empty((n_seqs, H, dk, dv), dtype=torch.float32, device=q.device)
    ck = torch.empty((max(int(max_checkpoints), 1), H, dk, dv), dtype=torch.float32,
                     device=q.device)[:int(max_checkpoints)]
    _check(load().kda_chunk_fwd_checkpoints(
        _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0), _ptr(cu_seqlens),
        _ptr(out), _ptr(S_final), T, n_seqs, H, dk, dv, int(interval),
        _ptr(ck) if int(max_checkpoints) > 0 else None, int(max_checkpoints), _stream(stream)))
    return out, S_final, ck


def kda_chunk_fwd_host(q, k, v, log_alpha, beta, S0, out, S_final, *, n_seqs, slice_tokens=0,
                       stream=None):
    """Prefill of a uniform batch held in HOST tensors (pin them for overlap).

    q, k, v, log_alpha, beta, out, S0 / S_final as in :func:`kda_chunk_fwd`, but CPU
    tensors; out and S_final are written once ``stream`` is synchronised."""
    T, H, dk = q.shape
    dv = v.shape[-1]
    for t, dt, name in ((q, torch.bfloat16, "q"), (k, torch.bfloat16, "k"),
                        (v, torch.bfloat16, "v"), (log_alpha, torch.float32, "log_alpha"),
                        (beta, torch.float32, "beta"), (S0, torch.float32, "S0"),
                        (out, torch.bfloat16, "out"), (S_final, torch.float32, "S_final")):
        if t is None:
            continue
        if t.is_cuda or t.dtype != dt or not t.is_contiguous():
            raise KdaError(1, f"{name} must be a contiguous CPU {dt} tensor")
    _check(load().kda_chunk_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                     _ptr(S0), _ptr(out), _ptr(S_final), T, n_seqs, H, dk, dv,
                                     int(slice_tokens), _stream(stream)))
    return out, S_final


def kda_decode_tokens_fused(q_raw, k_raw, v, gate, beta, S_inout, commit=None, out=None, *,
                            stream=None):
    """:func:`kda_decode_tokens` with raw q, k and bf16 gate logits [N, K, H, dk]."""
    N, K, H, dk = q_raw.shape
    dv = v.shape[-1]
    for t, dt, name in ((q_raw, torch.bfloat16, "q_raw"), (k_raw, torch.bfloat16, "k_raw"),
                        (v, torch.bfloat16, "v"), (gate, torch.bfloat16, "gate"),
                        (beta, torch.float32, "beta"), (S_inout, torch.float32, "S_inout"),
                        (commit, torch.int32, "commit")):
        _require(t, dt, name)
    if out is None:
        out = torch.empty((N, K, H, dv), dtype=torch.bfloat16, device=q_raw.device)
    _require(out, torch.bfloat16, "out")
    _check(load().kda_decode_tokens_fused(_ptr(q_raw), _ptr(k_raw), _ptr(v), _ptr(gate),
                                          _ptr(beta), _ptr(S_inout), _ptr(out), _ptr(commit),
                                          N, K, H, dk, dv, _stream(stream)))
    return out


# ---- operators around the recurrent layer.  Tensors may be column slices of wider ones: rows
# with a unit last stride, any row stride (over all leading dimensions).  Outputs that are not
# given are allocated on the call's stream.  All tensors of a call, and its stream, are on one
# GPU, which need not be the current one.

def _ops():
    """The module of csrc/kda_torch.cpp, its calls going to the library that load() returns."""
    global _extension, _selected
    load()
    with _lock:
        if _extension is None:
            if not os.path.exists(_EXT):
                failure = _finish_extension(_build_extension())
                if failure:
                    raise RuntimeError(f"kda_torch: {failure}")
            spec = importlib.util.spec_from_file_location("kda_torch", _EXT)
            _extension = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(_extension)
        _extension.select(library_path(), KdaError)
        _selected = _extension
    return _selected


def _call(stream, name, *args):
    f = getattr(_selected or _ops(), name)
    if stream is None:
        return f(*args)
    x = args[0]
    if isinstance(x, torch.Tensor) and x.is_cuda and x.device != stream.device:
        raise KdaError(1, f"the stream is on {stream.device}, the tensors on {x.device}")
    with torch.cuda.stream(stream):  # its outputs too belong to that stream
        return f(*args)


def kda_add_rms_norm(x, weight, residual=None, *, eps=1e-6, y=None, h=None, stream=None):
    """The residual's addition and the root-mean-square norm of the rows of x.

    x, residual: bf16 or f32 [..., dim], rows may be strided; weight: bf16 or f32 [dim].
    Returns (y, h): h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight, both in x's
    dtype; h is None without a residual (unless given).  y and h may be x or the residual.
    """
    y, _, h = _call(stream, "add_rms_norm", x, weight, residual, eps, y, None, h, False)
    return y, h


def kda_add_rms_norm_quant(x, weight, residual=None, *, eps=1e-6, y=None, y_scale=None, h=None,
                           stream=None):
    """:func:`kda_add_rms_norm` with y in 8 bits: returns (y, y_scale, h), y float8_e4m3fn
    [..., dim] and y_scale f32 [..., ceil(dim / 128)] with y * y_scale (per 128 columns)
    standing for the normalised rows, as :func:`kda_matmul_fp8` reads them."""
    return _call(stream, "add_rms_norm", x, weight, residual, eps, y, y_scale, h, True)


def kda_matmul_fp8(a, a_scale, b, b_scale, out=None, *, out_dtype=torch.bfloat16, stream=None):
    """a [..., K] times the transpose of b [N, K], both float8_e4m3fn with rows on 16-byte
    boundaries; a_scale: f32 [..., ceil(K / 128)], b_scale: f32 [ceil(N / 128), ceil(K / 128)].
    Returns out [..., N], rounded once from 32-bit sums: ``out``, or a new tensor of
    ``out_dtype`` (bf16 or f32)."""
    if out is None and out_dtype not in (torch.bfloat16, torch.float32):
        raise KdaError(1, f"out must be bfloat16 or float32, got {out_dtype}")
    return _call(stream, "matmul_fp8", a, a_scale, b, b_scale, out, out_dtype == torch.float32)


def kda_short_conv_fwd(x, weight, bias=None, conv_state=None, cu_seqlens=None, *, n_seqs=None,
                       silu=True, want_state=True, y=None, state_out=None, stream=None):
    """Short causal convolution per channel over packed sequences.

    x: bf16 or f32 [T, dim] (or [B, T_b, dim], a uniform batch), rows may be strided; weight:
    bf16 or f32 [dim, width]; bias: [dim] in weight's dtype or None; conv_state: [N, width - 1,
    dim] in x's dtype or None (zeros); cu_seqlens: int32 [N + 1] (CUDA) or None.  Returns
    (y, state): the state continues the sequences; ``state_out`` may be ``conv_state`` itself.
    """
    return _call(stream, "short_conv_fwd", x, weight, bias, conv_state, cu_seqlens, n_seqs,
                 bool(silu), bool(want_state), y, state_out)


def kda_short_conv_step(x, weight, conv_state, bias=None, *, silu=True, y=None, stream=None):
    """One token of each sequence: x [N, dim]; ``conv_state`` [N, width - 1, dim] is updated in
    place.  Otherwise as :func:`kda_short_conv_fwd`.  Returns y [N, dim]."""
    return _call(stream, "short_conv_step", x, weight, conv_state, bias, bool(silu), y)


def kda_ssm_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, *,
                     n_seqs=None, softplus=True, want_state=True, y=None, h_final=None,
                     stream=None):
    """Selective state space scan over packed sequences (see include/kda.h).

    x, dt, z: bf16 or f32 [T, dim] (or [B, T_b, dim], a uniform batch), rows may be strided;
    A: f32 [dim, state], negative; B, C: [T, groups, state] in x's dtype; D, dt_bias: f32 [dim]
    or None; h0: f32 [N, dim, state] or None (zeros); cu_seqlens: int32 [N + 1] (CUDA) or None.
    Returns (y, h_final); ``h_final`` may be ``h0`` itself.
    """
    return _call(stream, "ssm_scan_fwd", x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, n_seqs,
                 bool(softplus), bool(want_state), y, h_final)


def kda_ssm_scan_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, *, softplus=True, y=None,
                      stream=None):
    """One token of each sequence: x, dt, z [N, dim], B, C [N, groups, state]; ``h`` f32
    [N, dim, state] is updated in place.  Otherwise as :func:`kda_ssm_scan_fwd`.  Returns y."""
    return _call(stream, "ssm_scan_step", x, dt, A, B, C, h, D, z, dt_bias, bool(softplus), y)


# ---- full attention and its cache in 4 bits

def kda_attention_fwd(q, k, v, cu_seqlens_q=None, cu_seqlens_k=None, *, n_seqs=None, causal=True,
                      scale=None, want_lse=False, out=None, lse=None, stream=None):
    """Attention over prompts (see include/kda.h).

    q: bf16 [Tq, heads, d] (or [B, Tq_b, heads, d], a uniform batch); k, v: bf16 [Tk, kv_heads, d]
    (or [B, Tk_b, kv_heads, d]); a token's heads are dense, tokens may be any multiple of 16 bytes
    apart; cu_seqlens_q: int32 [N + 1] (CUDA) or None; cu_seqlens_k: the same for keys, None where
    they are the queries'.  With fewer queries than keys the queries are their sequence's last ones.
    scale: 1 / sqrt(d) if None.  Returns (out, lse): out as q, lse f32 [Tq, heads] (the logarithms
    of the sums) or None unless wanted or given.  n_seqs: the sequences of packed tokens of equal
    lengths (without cu_seqlens; a uniform batch has B).
    """
    return _call(stream, "attention_fwd", q, k, v, cu_seqlens_q, cu_seqlens_k, n_seqs, bool(causal),
                 scale, bool(want_lse), out, lse)


def kda_kv4_cache(n_pages, page_size, kv_heads, d, device="cuda"):
    """The arrays of a paged cache in 4 bits (layout: include/kda.h): (k_codes, k_scales, v_codes,
    v_scales), uint8 [n_pages, kv_heads, page_size, d / 2] and bf16 [.., d / 32], of zeros."""
    new = lambda n, dtype: torch.zeros(n_pages, kv_heads, page_size, n, dtype=dtype, device=device)
    codes, scales = (d // 2, torch.uint8), (d // 32, torch.bfloat16)
    return new(*codes), new(*scales), new(*codes), new(*scales)


def kda_kv4_write(k, v, cache, block_table, start=None, cu_seqlens=None, *, n_seqs=None, stream=None):
    """Quantise tokens into a paged cache (see include/kda.h), which is updated in place.

    k, v: bf16 [T, kv_heads, d] or [B, T_b, kv_heads, d]; cache: as :func:`kda_kv4_cache` makes it;
    block_table: int32 [N, max_pages], the pages of each sequence; start: int32 [N], the position of
    each sequence's first token (None: 0; negative: that sequence is left out); cu_seqlens: int32
    [N + 1] or None (N = block_table's rows, or ``n_seqs``, of equal length; B is N).
    """
    _call(stream, "kv4_write", k, v, cache, block_table, start, cu_seqlens, n_seqs)


def kda_kv4_read(cache, block_table, total_tokens, start=None, cu_seqlens=None, *, n_seqs=None, k=None,
                 v=None, stream=None):
    """Read positions of a paged cache back: the reverse of :func:`kda_kv4_write`.  Returns (k, v),
    bf16 [total_tokens, kv_heads, d]; rows of sequences that are left out stay as they are."""
    if stream is not None and isinstance(block_table, torch.Tensor) and block_table.is_cuda \
            and block_table.device != stream.device:
        raise KdaError(1, f"the stream is on {stream.device}, the tensors on {block_table.device}")
    return _call(stream, "kv4_read", cache, block_table, total_tokens, start, cu_seqlens, n_seqs, k, v)


def kda_kv4_attention(q, cache, block_table, seq_lens, *, scale=None, want_lse=False, out=None, lse=None,
                      stream=None):
    """Attention of each sequence's last tokens over a paged cache in 4 bits (see include/kda.h).

    q: bf16 [N, heads, d], or [N, n_tokens, heads, d] for several tokens of each sequence; seq_lens:
    int32 [N], the positions in the cache, the queries' own among them; cache and block_table as for
    :func:`kda_kv4_write`.  scale: 1 / sqrt(d) if None.  Returns (out, lse) as
    :func:`kda_attention_fwd`.
    """
    return _call(stream, "kv4_attention", q, cache, block_table, seq_lens, scale, bool(want_lse), out, lse)
