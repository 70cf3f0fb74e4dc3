"""Python binding of libspecverify (GB300 speculative-decoding verification).

Argument marshalling only: every step of the verification runs in the CUDA
kernels of ``libspecverify.so`` (built in-tree by ``build.py``). PyTorch is
used for device memory and streams. There is no CPU fallback: if the library
is missing or no CUDA device is present the calls raise.

Entry points (same names as the C ABI in ``include/specverify.h``):

* ``verify``         modified rejection sampling with temperature / top-k / top-p
* ``verify_tree``    greedy exact-match verification of a REST draft tree
* ``verify_mentor``  the lossy, KL-bounded mentor variant
* ``sample``         one draw per row from the transformed distribution
* ``token_logprobs`` log probabilities, ranks, entropies, likeliest alternatives
* ``tree_attention`` attention of the drafted nodes over a paged cache
* ``rotary``, ``cache_append_rotary``
                     the same append with rotary positions, queries rotated
* ``cache_weigh``, ``cache_evict``
                     accepted rows' attention weights added up, and the
                     positions of the least weight evicted
* ``cache_append``, ``cache_compact``, ``cache_resize``, ``cache_fork``
                     the paged cache itself, changed in place

Tensors may live on the GPU (the normal case) or in (pinned) host memory; host
inputs are copied to the current device, and outputs come back to the host.
A paged cache, its page table and its reference counts live on the GPU; a call
runs on their device, whichever is current.
"""

import collections
import contextlib
import ctypes
import functools
import inspect
import math
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")
# the same library built with device-side index checks (build.py --debug)
DEBUG_LIB_PATH = os.path.join(_HERE, "libspecverify_debug.so")

SPEC_OK, SPEC_EINVAL, SPEC_ECUDA, SPEC_ETIMEOUT, SPEC_EDATA, SPEC_EBOUNDS, SPEC_ENOPAGES = 0, 1, 2, 3, 4, 5, 6
SPEC_F32, SPEC_BF16 = 0, 1
MAX_TREE_N = 1024
MAX_TOP = 32
PURPOSE_ACCEPT, PURPOSE_RESAMPLE, PURPOSE_DRAFT = 0, 1, 2

EXPORTED = [
    "spec_verify_workspace_size", "spec_verify", "spec_verify_lenient",
    "spec_verify_tree_workspace_size", "spec_verify_tree", "spec_tree_build", "spec_acceptance_rate",
    "spec_expected_tokens", "spec_walltime_factor", "spec_ops_factor", "spec_best_gamma",
    "spec_verify_mentor_workspace_size", "spec_verify_mentor",
    "spec_sample_workspace_size", "spec_sample", "spec_token_logprobs",
    "spec_tree_attention_workspace_size", "spec_tree_attention", "spec_cache_append", "spec_cache_compact",
    "spec_rotary_turns", "spec_cache_append_rotary", "spec_cache_weigh", "spec_cache_evict_workspace_size",
    "spec_cache_evict",
    "spec_cache_resize", "spec_cache_fork_workspace_size", "spec_cache_fork",
    "spec_philox_uniform", "spec_verify_noalloc", "spec_status_string", "spec_last_cuda_error",
    "spec_version", "spec_debug_build", "spec_debug_failures", "spec_debug_withhold_copy", "spec_debug_withhold_tile",
]


class SpecSampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_p", ctypes.c_float), ("top_k", ctypes.c_int32)]


class SpecCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("layers", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("page_refs", ctypes.c_void_p)]


class _CacheArg:
    """A spec_cache argument: its packed bytes, or a SpecCache."""

    @staticmethod
    def from_param(x):
        return x if isinstance(x, bytes) else ctypes.byref(x)


class SpecError(RuntimeError):
    pass


_libs = {}
_current = [LIB_PATH]
_lock = threading.Lock()
_P = ctypes.c_void_p
_I = ctypes.c_int
_U64 = ctypes.c_uint64
_SZ = ctypes.c_size_t


def load_library(path=None):
    """Load the library (default: the one ``use_library`` selected, normally
    libspecverify.so) and declare its C signatures (no CUDA call)."""
    with _lock:
        path = path or _current[0]
        lib = _libs.get(path)
        if lib is not None:
            return lib
        if not os.path.exists(path):
            raise SpecError(f"{path} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(path)
        lib.spec_verify_workspace_size.argtypes = [_I, _I, _I, _I]
        lib.spec_verify_workspace_size.restype = _SZ
        lib.spec_verify.argtypes = [_P, _P, _I, _P, _I, _I, _I, SpecSampling, _U64, _U64,
                                    _P, _P, _P, _P, _P, _P, _SZ, _P]
        lib.spec_verify.restype = _I
        lib.spec_verify_lenient.argtypes = [_P, _P, _I, _P, _I, _I, _I, SpecSampling, ctypes.c_float, _U64, _U64,
                                            _P, _P, _P, _P, _P, _P, _SZ, _P]
        lib.spec_verify_lenient.restype = _I
        lib.spec_verify_tree_workspace_size.argtypes = [_I, _I, _I, _I]
        lib.spec_verify_tree_workspace_size.restype = _SZ
        lib.spec_verify_tree.argtypes = [_P, _I, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P,
                                         _P, _SZ, _P]
        lib.spec_verify_tree.restype = _I
        lib.spec_tree_build.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]
        lib.spec_tree_build.restype = _I
        lib.spec_acceptance_rate.argtypes = [_P, _P, _I, _I, _I, _I, SpecSampling, _P, _P, _P, _SZ, _P]
        lib.spec_acceptance_rate.restype = _I
        _D = ctypes.c_double
        lib.spec_expected_tokens.argtypes = [_D, _I]
        lib.spec_expected_tokens.restype = _D
        lib.spec_walltime_factor.argtypes = [_D, _I, _D]
        lib.spec_walltime_factor.restype = _D
        lib.spec_ops_factor.argtypes = [_D, _I, _D]
        lib.spec_ops_factor.restype = _D
        lib.spec_best_gamma.argtypes = [_D, _D, _I]
        lib.spec_best_gamma.restype = _I
        lib.spec_verify_mentor_workspace_size.argtypes = [_I, _I, _I, _I]
        lib.spec_verify_mentor_workspace_size.restype = _SZ
        lib.spec_verify_mentor.argtypes = [_P, _P, _I, _P, _I, _I, _I, ctypes.c_float, ctypes.c_float,
                                           _I, _U64, _U64, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        lib.spec_verify_mentor.restype = _I
        lib.spec_sample_workspace_size.argtypes = [_I, _I, _I, _I]
        lib.spec_sample_workspace_size.restype = _SZ
        lib.spec_sample.argtypes = [_P, _I, _I, _I, _I, SpecSampling, _U64, _U64, ctypes.c_uint32,
                                    ctypes.c_uint32, _P, _P, _P, _SZ, _P]
        lib.spec_sample.restype = _I
        lib.spec_token_logprobs.argtypes = [_P, _I, _P, _I, _I, _I, ctypes.c_float, _I, _P, _P, _P, _P, _P, _P, _P]
        lib.spec_token_logprobs.restype = _I
        lib.spec_verify_noalloc.argtypes = [_P, _P, _I, _P, _I, _I, _I, SpecSampling, _U64, _U64,
                                            _P, _P, _P, _P, _P, _P]
        lib.spec_verify_noalloc.restype = _I
        lib.spec_philox_uniform.argtypes = [_U64, _U64, ctypes.c_uint32, ctypes.c_uint32, _I, _P, _P]
        lib.spec_philox_uniform.restype = _I
        _C, _I64 = _CacheArg, ctypes.c_int64
        lib.spec_tree_attention_workspace_size.argtypes = [_I] * 6
        lib.spec_tree_attention_workspace_size.restype = _SZ
        lib.spec_tree_attention.argtypes = [_P, _C, _I, _P, _I64, _I, _P, _P, _P, _I, _I, _I, ctypes.c_float,
                                            _P, _P, _P, _P, _SZ, _P]
        lib.spec_tree_attention.restype = _I
        lib.spec_cache_append.argtypes = [_P, _P, _C, _I, _P, _I64, _I, _P, _P, _I, _I, _P, _P]
        lib.spec_cache_append.restype = _I
        lib.spec_rotary_turns.argtypes = [_I, _D, _I, _D, _D, ctypes.POINTER(_U64), ctypes.POINTER(ctypes.c_float)]
        lib.spec_rotary_turns.restype = _I
        lib.spec_cache_append_rotary.argtypes = [_P, _P, _P, _C, _I, _P, _I64, _I, _P, _P, _I, _I, ctypes.c_float, _P, _P,
                                                 _P, _I, _I, _I, _P, _P, _P]
        lib.spec_cache_append_rotary.restype = _I
        lib.spec_cache_compact.argtypes = [_C, _I, _P, _I64, _I, _P, _P, _P, _I, _I, _P, _P, _P]
        lib.spec_cache_compact.restype = _I
        lib.spec_cache_weigh.argtypes = [_P, _P, _C, _I, _P, _I64, _I, _P, _P, _P, _I, _I, _I, _I, ctypes.c_float, _P, _I64,
                                         _P, _P]
        lib.spec_cache_weigh.restype = _I
        lib.spec_cache_evict_workspace_size.argtypes = [_I, _I, _I, _I64]
        lib.spec_cache_evict_workspace_size.restype = _SZ
        lib.spec_cache_evict.argtypes = [_C, _I, _P, _I64, _I, _P, _P, _I, _I, _P, _I64, _I, _P, _P, _P, _SZ, _P]
        lib.spec_cache_evict.restype = _I
        lib.spec_cache_resize.argtypes = [_P, _I64, _I, _I, _P, _I, _I, _P, _P, _I, _P, _P]
        lib.spec_cache_resize.restype = _I
        lib.spec_cache_fork_workspace_size.argtypes = [_I]
        lib.spec_cache_fork_workspace_size.restype = _SZ
        lib.spec_cache_fork.argtypes = [_C, _I, _P, _I64, _I, _I, _P, _P, _P, _P, _I, _P, _P, _SZ, _P]
        lib.spec_cache_fork.restype = _I
        lib.spec_status_string.argtypes = [_I]
        lib.spec_status_string.restype = ctypes.c_char_p
        lib.spec_last_cuda_error.argtypes = []
        lib.spec_last_cuda_error.restype = ctypes.c_char_p
        lib.spec_version.argtypes = []
        lib.spec_version.restype = _I
        lib.spec_debug_build.argtypes = []
        lib.spec_debug_build.restype = _I
        lib.spec_debug_failures.argtypes = [_P]
        lib.spec_debug_failures.restype = _I
        lib.spec_debug_withhold_copy.argtypes = [_I]
        lib.spec_debug_withhold_copy.restype = _I
        lib.spec_debug_withhold_tile.argtypes = [_I]
        lib.spec_debug_withhold_tile.restype = _I
        _libs[path] = lib
        return lib


@contextlib.contextmanager
def use_library(path):
    """Route the calls of this module to the library at `path` (for example
    the debug build, DEBUG_LIB_PATH) inside the block."""
    load_library(path)
    with _lock:
        saved = _current[0]
        _current[0] = path
    try:
        yield
    finally:
        with _lock:
            _current[0] = saved


def _check(rc):
    if rc != SPEC_OK:
        lib = load_library()
        msg = lib.spec_status_string(rc).decode()
        if rc == SPEC_ECUDA:
            msg += ": " + lib.spec_last_cuda_error().decode()
        raise SpecError(msg)


def _device():
    return torch._C._cuda_getDevice()


def _on_device_of(name):
    """The call runs with the device of its tensor `name` current: a launch goes
    to the current device, and the default stream's handle is the same on all."""
    def wrap(fn):
        at = list(inspect.signature(fn).parameters).index(name)

        @functools.wraps(fn)
        def call(*args, **kw):
            try:
                index = (args[at] if len(args) > at else kw[name]).get_device()   # (a host tensor's is -1)
            except (AttributeError, KeyError):
                index = -1   # no tensor: the call says so itself
            if index < 0 or index == _device():
                return fn(*args, **kw)
            with torch.cuda.device(index):
                return fn(*args, **kw)
        return call
    return wrap


def _given(out, index, want):
    """The caller's output tensors as a new dict; each key's must be contiguous and
    on the call's device, with the shape and dtype that `want` has for it."""
    o = {} if out is None else dict(out)
    for key, (shape, dtype) in want.items():
        t = o.get(key)
        if t is not None and (t.dtype is not dtype or tuple(t.shape) != tuple(shape) or t.get_device() != index or
                              not t.is_contiguous()):
            raise SpecError(f"out[{key!r}] must be a contiguous {dtype} tensor {list(shape)} on the call's device")
    return o


def _dtype_code(t):
    if t.dtype == torch.float32:
        return SPEC_F32
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    raise SpecError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


_ws_cache = {}
_turns = {}


def _turn(index, raw):
    """The lock of a stream (device index, raw handle) under which a call takes its
    workspace and enqueues its kernels: they pass data through the workspace, so
    another thread's call on the stream must not come between them."""
    return _turns.get((index, raw)) or _turns.setdefault((index, raw), threading.Lock())


def workspace(nbytes, device, stream):
    """A workspace of at least nbytes, cached per (device, stream).

    The library clears what it needs at the start of every call, so the
    buffer is reused as is; calls on one stream never overlap on the GPU, and
    this module's calls enqueue all their kernels under the stream's lock. A
    call that a graph captures has a buffer of its own, from the graph's memory:
    a replay may come after the stream's buffer was replaced by a larger one, or
    beside calls on that stream.
    """
    if torch.cuda.is_current_stream_capturing():
        with torch.cuda.stream(stream):
            return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    key = (device.index if device.index is not None else torch.cuda.current_device(), stream.cuda_stream)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        with torch.cuda.stream(stream):
            buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


class _Staging:
    """Moves host inputs to the device and device outputs back (end-to-end calls)."""

    def __init__(self, ref):
        self.host = ref.device.type == "cpu"
        if self.host and not torch.cuda.is_available():
            raise SpecError("libspecverify needs a CUDA device; none is available")
        self.device = torch.device("cuda", torch.cuda.current_device()) if self.host else ref.device

    def dev(self, t, dtype=None):
        if t is None:
            return None
        if dtype is not None and t.dtype != dtype:
            t = t.to(dtype)
        if t.device != self.device:
            t = t.to(self.device, non_blocking=True)
        return t.contiguous()

    def out(self, shape, dtype=torch.int32):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def back(self, d):
        """Device outputs to host tensors: one asynchronous copy per output
        into a reused pinned buffer, one synchronisation, then copies into
        ordinary host tensors that the caller owns."""
        if not self.host:
            return d
        tens = {k: v for k, v in d.items() if isinstance(v, torch.Tensor)}
        total = sum(_al16(v.numel() * v.element_size()) for v in tens.values())
        with _pin_lock:
            buf = _pinned.get(self.device.index)
            if buf is None or buf.numel() < total:
                buf = torch.empty(max(total, 1 << 16), dtype=torch.uint8, pin_memory=True)
                _pinned[self.device.index] = buf
            views, o = {}, 0
            for k, v in tens.items():
                n = v.numel() * v.element_size()
                h = buf[o:o + n].view(v.dtype).view(v.shape)
                h.copy_(v, non_blocking=True)
                views[k] = h
                o += _al16(n)
            torch.cuda.current_stream(self.device).synchronize()
            res = {k: (views[k].clone() if k in views else v) for k, v in d.items()}
        return res


def _al16(n):
    return (n + 15) & ~15


_pinned = {}
_pin_lock = threading.Lock()


@_on_device_of("target")
def verify(target, draft, draft_tokens, temperature=1.0, top_p=1.0, top_k=0, seed=0, offset=0,
           debug=False, out=None, lenience=1.0):
    """Modified rejection sampling over target [B, gamma+1, V] and draft [B, gamma, V].

    Returns a dict of tensors: accepted [B], tokens [B, gamma+1], next_token [B],
    status [B] and, with debug=True, probs [B, gamma, 2] = (q(x_k), p(x_k)).
    ``out`` may pass preallocated output tensors under the same keys.
    ``lenience`` l < 1 selects spec_verify_lenient (acceptance min(1, q/(l p)),
    residual max(0, q - l p)); l = 1 is spec_verify.
    """
    lib = load_library()
    sg = _Staging(target)
    target = sg.dev(target)
    draft = sg.dev(draft) if (draft is not None and temperature != 0) else None
    toks = sg.dev(draft_tokens, torch.int32)
    B, G1, V = target.shape
    gamma = G1 - 1
    if toks.shape != (B, gamma) or (draft is not None and draft.shape != (B, gamma, V)):
        raise SpecError("shape mismatch between target, draft and draft_tokens")
    if draft is not None and draft.dtype != target.dtype:
        raise SpecError("target and draft must share a dtype")
    i32 = torch.int32
    o = _given(out, sg.device.index, {"accepted": ((B,), i32), "tokens": ((B, G1), i32), "next_token": ((B,), i32),
                                      "status": ((B,), i32), "probs": ((B, gamma, 2), torch.float32)})
    o.setdefault("accepted", sg.out((B,)))
    o.setdefault("tokens", sg.out((B, G1)))
    o.setdefault("next_token", sg.out((B,)))
    o.setdefault("status", sg.out((B,)))
    if debug:
        o.setdefault("probs", sg.out((B, gamma, 2), torch.float32))
    dt = _dtype_code(target)
    stream = torch.cuda.current_stream(sg.device)
    nbytes = lib.spec_verify_workspace_size(B, gamma, V, dt)
    smp = SpecSampling(float(temperature), float(top_p), int(top_k))
    with _turn(sg.device.index, stream.cuda_stream):
        ws = workspace(nbytes, sg.device, stream)
        outs = (_ptr(o["accepted"]), _ptr(o["tokens"]), _ptr(o["next_token"]), _ptr(o["status"]),
                _ptr(o.get("probs")), _ptr(ws), ws.numel(), ctypes.c_void_p(stream.cuda_stream))
        if lenience == 1.0:
            rc = lib.spec_verify(_ptr(target), _ptr(draft), dt, _ptr(toks), B, gamma, V, smp, int(seed), int(offset),
                                 *outs)
        else:
            rc = lib.spec_verify_lenient(_ptr(target), _ptr(draft), dt, _ptr(toks), B, gamma, V, smp,
                                         float(lenience), int(seed), int(offset), *outs)
    _check(rc)
    return sg.back(o)


@_on_device_of("target")
def verify_tree(target, node_tokens, parent, depth, max_depth):
    """Greedy exact-match verification of BFS-ordered draft trees [B, N, V].

    Returns accept_len [B], path_nodes [B, max_depth+1], tokens [B, max_depth+1],
    bonus [B], status [B].
    """
    lib = load_library()
    sg = _Staging(target)
    target = sg.dev(target)
    tok, par, dep = (sg.dev(t, torch.int32) for t in (node_tokens, parent, depth))
    B, N, V = target.shape
    W = max_depth + 1
    o = {"accept_len": sg.out((B,)), "path_nodes": sg.out((B, W)), "tokens": sg.out((B, W)),
         "bonus": sg.out((B,)), "status": sg.out((B,))}
    dt = _dtype_code(target)
    stream = torch.cuda.current_stream(sg.device)
    with _turn(sg.device.index, stream.cuda_stream):
        ws = workspace(lib.spec_verify_tree_workspace_size(B, N, V, dt), sg.device, stream)
        rc = lib.spec_verify_tree(_ptr(target), dt, _ptr(tok), _ptr(par), _ptr(dep), B, N, V, int(max_depth),
                                  _ptr(o["accept_len"]), _ptr(o["path_nodes"]), _ptr(o["tokens"]),
                                  _ptr(o["bonus"]), _ptr(o["status"]), _ptr(ws), ws.numel(),
                                  ctypes.c_void_p(stream.cuda_stream))
    _check(rc)
    return sg.back(o)


@_on_device_of("candidates")
def tree_build(candidates, root_token, V, N, counts=None, with_mask=True):
    """REST draft trees from retrieved continuations candidates [B, C, L] (-1 ends one).

    Returns node_tokens, parent, depth [B, N] (the layout ``verify_tree`` takes),
    mask [B, N, N] uint8 (when ``with_mask``), n_nodes [B] and status [B].
    """
    lib = load_library()
    sg = _Staging(candidates)
    cand = sg.dev(candidates, torch.int32)
    root = sg.dev(root_token, torch.int32)
    cnt = sg.dev(counts, torch.int32)
    B, C, L = cand.shape
    o = {"node_tokens": sg.out((B, N)), "parent": sg.out((B, N)), "depth": sg.out((B, N)),
         "n_nodes": sg.out((B,)), "status": sg.out((B,))}
    if with_mask:
        o["mask"] = sg.out((B, N, N), torch.uint8)
    stream = torch.cuda.current_stream(sg.device)
    rc = lib.spec_tree_build(_ptr(cand), _ptr(cnt), _ptr(root), B, C, L, int(V), int(N),
                             _ptr(o["node_tokens"]), _ptr(o["parent"]), _ptr(o["depth"]), _ptr(o.get("mask")),
                             _ptr(o["n_nodes"]), _ptr(o["status"]), ctypes.c_void_p(stream.cuda_stream))
    _check(rc)
    return sg.back(o)


@_on_device_of("target")
def acceptance_rate(target, draft, temperature=1.0, top_p=1.0, top_k=0):
    """beta [B, gamma] = sum_x min(q_k(x), p_k(x)) per position (temperature > 0),
    and status [B]; the mean of beta estimates the acceptance rate alpha."""
    lib = load_library()
    sg = _Staging(target)
    target, draft = sg.dev(target), sg.dev(draft)
    B, G1, V = target.shape
    gamma = G1 - 1
    if draft.shape != (B, gamma, V) or draft.dtype != target.dtype:
        raise SpecError("shape or dtype mismatch between target and draft")
    o = {"beta": sg.out((B, gamma), torch.float32), "status": sg.out((B,))}
    dt = _dtype_code(target)
    stream = torch.cuda.current_stream(sg.device)
    with _turn(sg.device.index, stream.cuda_stream):
        ws = workspace(lib.spec_verify_workspace_size(B, gamma, V, dt), sg.device, stream)
        rc = lib.spec_acceptance_rate(_ptr(target), _ptr(draft), dt, B, gamma, V,
                                      SpecSampling(float(temperature), float(top_p), int(top_k)),
                                      _ptr(o["beta"]), _ptr(o["status"]), _ptr(ws), ws.numel(),
                                      ctypes.c_void_p(stream.cuda_stream))
    _check(rc)
    return sg.back(o)


def expected_tokens(alpha, gamma):
    """E[#tokens per target call] for acceptance rate alpha and draft length gamma."""
    return load_library().spec_expected_tokens(float(alpha), int(gamma))


def walltime_factor(alpha, gamma, c):
    """Expected walltime improvement for draft cost ratio c."""
    return load_library().spec_walltime_factor(float(alpha), int(gamma), float(c))


def ops_factor(alpha, gamma, c_hat):
    """Expected factor on the total number of operations."""
    return load_library().spec_ops_factor(float(alpha), int(gamma), float(c_hat))


def best_gamma(alpha, c, gamma_max):
    """The draft length in 1..gamma_max with the largest walltime factor."""
    return load_library().spec_best_gamma(float(alpha), float(c), int(gamma_max))


@_on_device_of("target")
def verify_mentor(target, draft, draft_tokens, temperature=1.0, kl_bound=0.0, bisect_iters=30,
                  seed=0, offset=0, debug=False):
    """Lossy mentor verification; returns the ``verify`` outputs plus alpha and beta [B, gamma]."""
    lib = load_library()
    sg = _Staging(target)
    target, draft = sg.dev(target), sg.dev(draft)
    toks = sg.dev(draft_tokens, torch.int32)
    B, G1, V = target.shape
    gamma = G1 - 1
    if draft.shape != (B, gamma, V) or toks.shape != (B, gamma) or draft.dtype != target.dtype:
        raise SpecError("shape or dtype mismatch between target, draft and draft_tokens")
    o = {"accepted": sg.out((B,)), "tokens": sg.out((B, G1)), "next_token": sg.out((B,)),
         "status": sg.out((B,)), "alpha": sg.out((B, gamma), torch.float32),
         "beta": sg.out((B, gamma), torch.float32)}
    if debug:
        o["probs"] = sg.out((B, gamma, 2), torch.float32)
    dt = _dtype_code(target)
    stream = torch.cuda.current_stream(sg.device)
    with _turn(sg.device.index, stream.cuda_stream):
        ws = workspace(lib.spec_verify_mentor_workspace_size(B, gamma, V, dt), sg.device, stream)
        rc = lib.spec_verify_mentor(_ptr(target), _ptr(draft), dt, _ptr(toks), B, gamma, V,
                                    float(temperature), float(kl_bound), int(bisect_iters), int(seed),
                                    int(offset), _ptr(o["accepted"]), _ptr(o["tokens"]),
                                    _ptr(o["next_token"]), _ptr(o["status"]), _ptr(o["alpha"]),
                                    _ptr(o["beta"]), _ptr(o.get("probs")), _ptr(ws), ws.numel(),
                                    ctypes.c_void_p(stream.cuda_stream))
    _check(rc)
    return sg.back(o)


@_on_device_of("logits")
def sample(logits, temperature=1.0, top_p=1.0, top_k=0, seed=0, offset=0, pos0=0,
           purpose=PURPOSE_DRAFT):
    """One draw per row of logits [B, P, V]; returns tokens [B, P] and status [B]."""
    lib = load_library()
    sg = _Staging(logits)
    logits = sg.dev(logits)
    B, P, V = logits.shape
    o = {"tokens": sg.out((B, P)), "status": sg.out((B,))}
    dt = _dtype_code(logits)
    stream = torch.cuda.current_stream(sg.device)
    with _turn(sg.device.index, stream.cuda_stream):
        ws = workspace(lib.spec_sample_workspace_size(B, P, V, dt), sg.device, stream)
        rc = lib.spec_sample(_ptr(logits), dt, B, P, V, SpecSampling(float(temperature), float(top_p), int(top_k)),
                             int(seed), int(offset), int(pos0), int(purpose), _ptr(o["tokens"]),
                             _ptr(o["status"]), _ptr(ws), ws.numel(), ctypes.c_void_p(stream.cuda_stream))
    _check(rc)
    return sg.back(o)


@_on_device_of("logits")
def token_logprobs(logits, tokens, top=0, temperature=1.0):
    """Log probabilities of tokens [B, P] under softmax(logits [B, P, V] / temperature).

    Token -1 marks a row that has none and is not read: ``verify``'s tokens go
    with its target as they are. Returns logprob [B, P] (0 where there is no
    token), rank [B, P] (tokens before it by logit, then by index; -1), entropy
    [B, P] in nats (0), status [B] and, with ``top`` <= 32, the likeliest
    top_tokens and top_logprobs [B, P, top] (-1, -inf). A row with NaN or +inf,
    or only -inf, or a token outside the vocabulary gives NaN and -1 and its
    sequence SPEC_EDATA.
    """
    lib = _library()
    host = not logits.is_cuda
    sg = _Staging(logits) if host else None
    dev = sg.device if host else logits.device
    index = dev.index
    dt = _dtype_code(logits)
    if logits.dim() != 3:
        raise SpecError("logits must be [B, P, V]")
    B, P, V = logits.shape
    if tokens.shape != (B, P):
        raise SpecError("tokens must be [B, P]")
    if not 0 <= top <= min(V, MAX_TOP):
        raise SpecError(f"top must be in 0 .. min(V, {MAX_TOP})")
    logits = sg.dev(logits) if host else logits.contiguous()
    tokens = _in(tokens, dev, index)
    f32, i32 = dict(dtype=torch.float32, device=dev), dict(dtype=torch.int32, device=dev)
    o = {"logprob": torch.empty((B, P), **f32), "rank": torch.empty((B, P), **i32),
         "entropy": torch.empty((B, P), **f32), "status": torch.empty((B,), **i32)}
    if top:
        o["top_tokens"], o["top_logprobs"] = torch.empty((B, P, top), **i32), torch.empty((B, P, top), **f32)
    rc = lib.spec_token_logprobs(logits.data_ptr(), dt, tokens.data_ptr(), B, P, V, temperature, top,
                                 o["logprob"].data_ptr(), o["rank"].data_ptr(), o["entropy"].data_ptr(),
                                 o["top_tokens"].data_ptr() if top else None,
                                 o["top_logprobs"].data_ptr() if top else None, o["status"].data_ptr(),
                                 _raw_stream(index))
    if rc:
        _check(rc)
    return sg.back(o) if host else o


def philox_uniform(seed, row0, position, purpose, n, device=None):
    """The library's uniforms U(seed, row0 + i, position, purpose), i < n (device float32)."""
    lib = load_library()
    device = device or torch.device("cuda", torch.cuda.current_device())
    out = torch.empty(n, dtype=torch.float32, device=device)
    stream = torch.cuda.current_stream(device)
    with torch.cuda.device(device):
        _check(lib.spec_philox_uniform(int(seed), int(row0), int(position), int(purpose), int(n), _ptr(out),
                                       ctypes.c_void_p(stream.cuda_stream)))
    return out


# ---- the paged key / value cache --------------------------------------------------
#
# These calls run once a layer and step, so the host side is kept short: plain
# attribute reads, one packed struct, integer pointers, cached workspace sizes.

_pack_cache = struct.Struct("@QQiiiii4xqqqqQ").pack   # spec_cache
_LIVE = {torch.float32: SPEC_F32, torch.bfloat16: SPEC_BF16}


def _library():
    return _libs.get(_current[0]) or load_library()


def _raw_stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


def _scratch(nbytes, dev, index, raw):
    """As ``workspace``, by the stream's raw handle (the same buffers)."""
    buf = _ws_cache.get((index, raw))
    if buf is None or buf.numel() < nbytes or torch.cuda.is_current_stream_capturing():
        buf = workspace(nbytes, dev, torch.cuda.current_stream(dev))
    return buf


def _cache_args(k_cache, v_cache, layered, page_refs=None):
    """The packed spec_cache of k / v caches [layers, pages, page_size, heads, head_dim]
    (one layer: no first dimension; any strides with contiguous heads), its
    shape and its dtype code."""
    sh, st = k_cache.shape, k_cache.stride()
    if len(sh) != 4 + layered or v_cache.shape != sh or v_cache.dtype != k_cache.dtype:
        raise SpecError("k and v caches must share a dtype and the shape "
                        + ("[layers, " if layered else "[") + "pages, page_size, heads, head_dim]")
    if v_cache.stride() != st or st[-1] != 1:
        raise SpecError("k and v caches must share their strides, with contiguous heads")
    if not k_cache.is_cuda or v_cache.get_device() != k_cache.get_device():
        raise SpecError("the caches must be on one CUDA device")
    dt = _LIVE.get(k_cache.dtype)
    if dt is None:
        raise SpecError(f"caches must be float32 or bfloat16, got {k_cache.dtype}")
    refs = 0 if page_refs is None else _owned(page_refs, (sh[-4],), k_cache.get_device(), "page_refs")
    return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), sh[0] if layered else 1, sh[-4], sh[-3], sh[-2], sh[-1],
                       st[0] if layered else 0, st[-4], st[-3], st[-2], refs), sh, dt


def _table_args(page_table, rows, index):
    """Pointer, row stride and width of an int32 page table with `rows` rows."""
    sh = page_table.shape
    if len(sh) != 2 or page_table.dtype is not torch.int32 or sh[0] != rows or page_table.get_device() != index or \
            (sh[1] > 1 and page_table.stride(1) != 1):
        raise SpecError(f"page_table must be an int32 tensor [{rows}, max_pages] on the cache's device, rows contiguous")
    # a single row's stride is free to be anything
    return page_table.data_ptr(), (page_table.stride(0) if rows > 1 else sh[1]), sh[1]


def _in(t, dev, index, dtype=torch.int32):
    """An input on the device in the library's layout (copied only if it is not there yet)."""
    if t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        # a view that starts off 16 bytes: rows are moved as 16-byte words
        return t.clone() if t.data_ptr() & 15 and t.is_floating_point() else t
    return _in(t.to(dtype).to(dev, non_blocking=True).contiguous(), dev, index, dtype)


def _owned(t, shape, index, what):
    if t.dtype is not torch.int32 or tuple(t.shape) != shape or t.get_device() != index or not t.is_contiguous():
        raise SpecError(f"{what} must be a contiguous int32 tensor {list(shape)} on the cache's device")
    return t.data_ptr()


@functools.lru_cache(maxsize=256)
def _attention_bytes(path, B, N, Hq, Hkv, D, dt):
    return load_library(path).spec_tree_attention_workspace_size(B, N, Hq, Hkv, D, dt)


@_on_device_of("k_cache")
def tree_attention(q, k_cache, v_cache, page_table, cache_len, mask=None, n_nodes=None, scale=None,
                   with_lse=False, out=None):
    """Attention of the drafted nodes q [B, N, heads, D] over one layer's cache.

    k_cache, v_cache [pages, page_size, kv_heads, D] (any strides with
    contiguous heads) hold the nodes' keys and values already (``cache_append``).
    Node i sees the cache_len[b] context positions and the nodes j < n_nodes[b]
    with mask[b, i, j] != 0 (``tree_build``'s mask; None: j <= i, a chain).
    ``scale`` defaults to 1 / sqrt(D). Returns out [B, N, heads, D], status [B]
    and, with ``with_lse``, lse [B, N, heads]; nodes from n_nodes[b] on are
    zero (lse -inf). ``out`` may pass preallocated outputs under these keys
    (contiguous, of these shapes and types, on the cache's device).
    """
    lib = _library()
    cache, sh, dt = _cache_args(k_cache, v_cache, 0)
    if q.dim() != 4 or q.shape[3] != sh[3] or q.shape[2] % sh[2] != 0 or q.dtype is not k_cache.dtype:
        raise SpecError("q must be [B, N, heads, head_dim] of the cache's dtype, heads a multiple of kv_heads")
    B, N, Hq, D = q.shape
    dev, index = k_cache.device, k_cache.get_device()
    table, stride, width = _table_args(page_table, B, index)
    host = not q.is_cuda
    q = _in(q, dev, index, q.dtype)
    lens = _in(cache_len, dev, index)
    if mask is not None:
        mask = _in(mask, dev, index, torch.uint8)
        if mask.shape != (B, N, N):
            raise SpecError("mask must be [B, N, N]")
    if n_nodes is not None:
        n_nodes = _in(n_nodes, dev, index)
    if lens.shape != (B,) or (n_nodes is not None and n_nodes.shape != (B,)):
        raise SpecError("cache_len and n_nodes must be [B]")
    o = {} if out is None else _given(out, index, {"out": (q.shape, q.dtype), "lse": ((B, N, Hq), torch.float32),
                                                   "status": ((B,), torch.int32)})
    if "out" not in o:
        o["out"] = torch.empty_like(q)
    if "status" not in o:
        o["status"] = torch.empty((B,), dtype=torch.int32, device=dev)
    if with_lse and "lse" not in o:
        o["lse"] = torch.empty((B, N, Hq), dtype=torch.float32, device=dev)
    raw = _raw_stream(index)
    with _turn(index, raw):
        ws = _scratch(_attention_bytes(_current[0], B, N, Hq, sh[2], D, dt), dev, index, raw)
        rc = lib.spec_tree_attention(q.data_ptr(), cache, dt, table, stride, width, lens.data_ptr(),
                                     None if mask is None else mask.data_ptr(),
                                     None if n_nodes is None else n_nodes.data_ptr(), B, N, Hq,
                                     D ** -0.5 if scale is None else scale, o["out"].data_ptr(),
                                     o["lse"].data_ptr() if "lse" in o else None, o["status"].data_ptr(),
                                     ws.data_ptr(), ws.numel(), raw)
    if rc:
        _check(rc)
    return {n: t.cpu() for n, t in o.items()} if host else o


@_on_device_of("k_cache")
def cache_append(k, v, k_cache, v_cache, page_table, cache_len, n_nodes=None, page_refs=None):
    """Write k, v [B, N, kv_heads, D] to positions cache_len[b] + i, i < n_nodes[b]
    (None: N), of one layer's cache [pages, page_size, kv_heads, D], in place.

    The pages must be the sequences' already (``cache_resize``) and nobody
    else's: with ``page_refs`` a sequence whose new rows would go to a shared
    page (it was shortened to inside one; ``cache_fork`` it instead) is refused,
    SPEC_EDATA. cache_len is not changed. Returns status [B].
    """
    lib = _library()
    cache, sh, dt = _cache_args(k_cache, v_cache, 0, page_refs)
    if k.dim() != 4 or k.shape != v.shape or k.shape[2:] != sh[2:] or k.dtype is not k_cache.dtype or \
            v.dtype is not k_cache.dtype:
        raise SpecError("k and v must be [B, N, kv_heads, head_dim] of the cache's dtype")
    B, N = k.shape[:2]
    dev, index = k_cache.device, k_cache.get_device()
    table, stride, width = _table_args(page_table, B, index)
    k, v, lens = _in(k, dev, index, k.dtype), _in(v, dev, index, v.dtype), _in(cache_len, dev, index)
    if n_nodes is not None:
        n_nodes = _in(n_nodes, dev, index)
    if lens.shape != (B,) or (n_nodes is not None and n_nodes.shape != (B,)):
        raise SpecError("cache_len and n_nodes must be [B]")
    status = torch.empty((B,), dtype=torch.int32, device=dev)
    rc = lib.spec_cache_append(k.data_ptr(), v.data_ptr(), cache, dt, table, stride, width, lens.data_ptr(),
                               None if n_nodes is None else n_nodes.data_ptr(), B, N, status.data_ptr(),
                               _raw_stream(index))
    if rc:
        _check(rc)
    return {"status": status}


Rotary = collections.namedtuple("Rotary", "turns interleaved factor")
Rotary.__doc__ = """Rotary frequencies on a device: turns [dim / 2] int64 (2^-64 of a turn a position), the pairs'
layout and the factor of cosine and sine. Made by ``rotary``, kept with the model."""
_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


def rotary(dim, base=10000.0, interleaved=False, scaling=None, scale=1.0, original=0.0, frequencies=None, device=None):
    """Rotary frequencies of the first ``dim`` columns of a head, for ``cache_append_rotary``.

    Pairs are columns (j, j + dim / 2) or, ``interleaved``, (2 j, 2 j + 1); pair j
    turns by base^(-2 j / dim) radians a position. ``scaling`` for long contexts:
    "linear" (frequencies divided by ``scale``), "ntk" (a larger base), "yarn" and
    "bands" (slow pairs divided, fast ones kept; ``original``: the length that the
    model was trained on). Or ``frequencies``: dim / 2 radians a position.
    """
    if scaling not in _SCALINGS:
        raise SpecError(f"scaling must be one of {list(_SCALINGS)}")
    if dim < 2 or dim % 2:
        raise SpecError("dim must be even and positive")
    factor, turns = ctypes.c_float(1.0), (_U64 * (dim // 2))()
    if frequencies is None:
        _check(load_library().spec_rotary_turns(dim, base, _SCALINGS[scaling], scale, original, turns, ctypes.byref(factor)))
    else:
        f = torch.as_tensor(frequencies, dtype=torch.float64).tolist()
        if scaling is not None or not isinstance(f, list) or len(f) != dim // 2 or not all(map(math.isfinite, f)):
            raise SpecError("frequencies must be dim / 2 finite numbers, without a scaling")
        turns[:] = [int(x / (2.0 * math.pi) % 1.0 * 2.0 ** 64) % 2 ** 64 for x in f]
    signed = [t - 2 ** 64 if t >= 2 ** 63 else t for t in turns]
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return Rotary(torch.tensor(signed, dtype=torch.int64, device=device), bool(interleaved), factor.value)


@_on_device_of("k_cache")
def cache_append_rotary(q, k, v, k_cache, v_cache, page_table, cache_len, rotary, positions=None, depth=None,
                        n_nodes=None, page_refs=None):
    """``cache_append`` with rotary positions: queries q [B, N, heads, D] rotated, keys
    k [B, N, kv_heads, D] rotated into the cache, values as they are.

    Node i is at position positions[b] + depth[b, i] of the text (``positions``
    [B], None: cache_len, which differs once ``cache_evict`` has shortened the
    cache; ``depth`` [B, N] ``tree_build``'s, None: i, a chain). ``rotary``: the
    frequencies (the function of this name). Returns q (rotated; zero from
    n_nodes[b] on) and status [B] as ``cache_append``.
    """
    lib = _library()
    cache, sh, dt = _cache_args(k_cache, v_cache, 0, page_refs)
    if k.dim() != 4 or k.shape != v.shape or k.shape[2:] != sh[2:] or k.dtype is not k_cache.dtype or \
            v.dtype is not k_cache.dtype:
        raise SpecError("k and v must be [B, N, kv_heads, head_dim] of the cache's dtype")
    B, N = k.shape[:2]
    if q.dim() != 4 or q.shape[:2] != (B, N) or q.shape[3] != sh[3] or q.dtype is not k_cache.dtype:
        raise SpecError("q must be [B, N, heads, head_dim] of the cache's dtype")
    dev, index = k_cache.device, k_cache.get_device()
    table, stride, width = _table_args(page_table, B, index)
    turns = rotary.turns
    if turns.dtype is not torch.int64 or turns.dim() != 1 or turns.get_device() != index or not turns.is_contiguous():
        raise SpecError("rotary must be of the cache's device (rotary(..., device=))")
    q, k, v = _in(q, dev, index, q.dtype), _in(k, dev, index, k.dtype), _in(v, dev, index, v.dtype)
    ints = [None if t is None else _in(t, dev, index) for t in (cache_len, positions, n_nodes)]
    if any(t is not None and t.shape != (B,) for t in ints):
        raise SpecError("cache_len, positions and n_nodes must be [B]")
    lens, positions, n_nodes = ints
    if depth is not None:
        depth = _in(depth, dev, index)
        if depth.shape != (B, N):
            raise SpecError("depth must be [B, N]")
    out = torch.empty_like(q)
    status = torch.empty((B,), dtype=torch.int32, device=dev)
    rc = lib.spec_cache_append_rotary(q.data_ptr(), k.data_ptr(), v.data_ptr(), cache, dt, table, stride, width,
                                      lens.data_ptr(), turns.data_ptr(), 2 * turns.shape[0], rotary.interleaved,
                                      rotary.factor, None if positions is None else positions.data_ptr(),
                                      None if depth is None else depth.data_ptr(),
                                      None if n_nodes is None else n_nodes.data_ptr(), B, N, q.shape[2],
                                      out.data_ptr(), status.data_ptr(), _raw_stream(index))
    if rc:
        _check(rc)
    return {"q": out, "status": status}


@_on_device_of("k_cache")
def cache_compact(k_cache, v_cache, page_table, cache_len, accept_len, path_nodes=None, page_refs=None):
    """Keep an accepted path in caches [layers, pages, page_size, kv_heads, D], in
    place: position L + i <- L + path_nodes[b, i], i <= accept_len[b].

    accept_len [B] and path_nodes [B, W] are ``verify_tree``'s; None: a chain
    (``verify``'s accepted), whose entries are in place. With ``page_refs`` a
    sequence whose entries would move into a shared page is refused. Returns
    cache_len [B] = L + accept_len + 1 (-1 on a data error) and status [B].
    """
    lib = _library()
    cache, _, dt = _cache_args(k_cache, v_cache, 1, page_refs)
    B = page_table.shape[0]
    dev, index = k_cache.device, k_cache.get_device()
    table, stride, width = _table_args(page_table, B, index)
    lens, acc = _in(cache_len, dev, index), _in(accept_len, dev, index)
    path = None if path_nodes is None else _in(path_nodes, dev, index)
    if lens.shape != (B,) or acc.shape != (B,) or (path is not None and (path.dim() != 2 or path.shape[0] != B)):
        raise SpecError("cache_len and accept_len must be [B], path_nodes [B, W]")
    new_len = torch.empty((B,), dtype=torch.int32, device=dev)
    status = torch.empty((B,), dtype=torch.int32, device=dev)
    rc = lib.spec_cache_compact(cache, dt, table, stride, width, lens.data_ptr(), acc.data_ptr(),
                                None if path is None else path.data_ptr(), B,
                                MAX_TREE_N if path is None else path.shape[1], new_len.data_ptr(), status.data_ptr(),
                                _raw_stream(index))
    if rc:
        _check(rc)
    return {"cache_len": new_len, "status": status}


def _weights(weights, shape, index):
    """Pointer and capacity of float32 weights shape + [capacity], changed in place."""
    sh = tuple(weights.shape)
    if weights.dtype is not torch.float32 or len(sh) != len(shape) + 1 or sh[:-1] != shape or \
            weights.get_device() != index or not weights.is_contiguous():
        raise SpecError(f"weights must be a contiguous float32 tensor {[*shape, 'capacity']} on the cache's device")
    return weights.data_ptr(), sh[-1]


@_on_device_of("k_cache")
def cache_weigh(q, lse, k_cache, page_table, cache_len, weights, accept_len=None, path_nodes=None, scale=None):
    """Add the accepted rows' attention weights to weights [B, kv_heads, capacity], in place:
    weights[b, g, t] += sum over rows r <= accept_len[b] with t <= L + r and the
    query heads of g of exp(scale q . k_t - lse).

    q [B, N, heads, D] and lse [B, N, heads] are ``tree_attention``'s (with_lse),
    k_cache one layer's, cache_len the length L before the step. Row r is node
    path_nodes[b, r] (``verify_tree``'s, after ``cache_compact``; None: r), and
    accept_len -1 .. the last row's number (None: all N rows of a chain). Returns
    status [B].
    """
    lib = _library()
    cache, sh, dt = _cache_args(k_cache, k_cache, 0)
    if q.dim() != 4 or q.shape[3] != sh[3] or q.shape[2] % sh[2] != 0 or q.dtype is not k_cache.dtype:
        raise SpecError("q must be [B, N, heads, head_dim] of the cache's dtype, heads a multiple of kv_heads")
    B, N, Hq, D = q.shape
    dev, index = k_cache.device, k_cache.get_device()
    table, stride, width = _table_args(page_table, B, index)
    w, capacity = _weights(weights, (B, sh[2]), index)
    q, z, lens = _in(q, dev, index, q.dtype), _in(lse, dev, index, torch.float32), _in(cache_len, dev, index)
    acc = None if accept_len is None else _in(accept_len, dev, index)
    path = None if path_nodes is None else _in(path_nodes, dev, index)
    if z.shape != (B, N, Hq):
        raise SpecError("lse must be [B, N, heads]")
    if lens.shape != (B,) or (acc is not None and acc.shape != (B,)) or \
            (path is not None and (acc is None or path.dim() != 2 or path.shape[0] != B)):
        raise SpecError("cache_len and accept_len must be [B], path_nodes (with accept_len) [B, W]")
    status = torch.empty((B,), dtype=torch.int32, device=dev)
    rc = lib.spec_cache_weigh(q.data_ptr(), z.data_ptr(), cache, dt, table, stride, width, lens.data_ptr(),
                              None if acc is None else acc.data_ptr(), None if path is None else path.data_ptr(), B, N,
                              N if path is None else path.shape[1], Hq, D ** -0.5 if scale is None else scale, w, capacity,
                              status.data_ptr(), _raw_stream(index))
    if rc:
        _check(rc)
    return {"status": status}


@_on_device_of("k_cache")
def cache_evict(k_cache, v_cache, page_table, cache_len, weights, budget, sink=0, recent=0, page_refs=None):
    """Shorten sequences of more than budget[b] positions to budget[b], in place, in
    caches [layers, pages, page_size, kv_heads, D]: every layer and head keeps its
    first ``sink``, its last ``recent`` and the heaviest positions between them by
    weights [layers, B, kv_heads, capacity] (``cache_weigh``'s of every layer), in
    their order.

    Weights move along, those past the new length become zero. ``budget``: [B], or
    a number for all. With ``page_refs`` a sequence whose entries would move into a
    shared page is refused. Returns cache_len [B] (-1 on a data error) and status
    [B]; ``cache_resize`` then releases the pages.
    """
    lib = _library()
    cache, sh, dt = _cache_args(k_cache, v_cache, 1, page_refs)
    B = page_table.shape[0]
    dev, index = k_cache.device, k_cache.get_device()
    table, stride, width = _table_args(page_table, B, index)
    w, capacity = _weights(weights, (sh[0], B, sh[3]), index)
    lens = _in(cache_len, dev, index)
    most = _in(budget, dev, index) if torch.is_tensor(budget) else torch.full((B,), budget, dtype=torch.int32, device=dev)
    if lens.shape != (B,) or most.shape != (B,):
        raise SpecError("cache_len and budget must be [B]")
    new_len = torch.empty((B,), dtype=torch.int32, device=dev)
    status = torch.empty((B,), dtype=torch.int32, device=dev)
    raw = _raw_stream(index)
    with _turn(index, raw):
        ws = _scratch(lib.spec_cache_evict_workspace_size(sh[0], B, sh[3], capacity), dev, index, raw)
        rc = lib.spec_cache_evict(cache, dt, table, stride, width, lens.data_ptr(), most.data_ptr(), sink, recent, w,
                                  capacity, B, new_len.data_ptr(), status.data_ptr(), ws.data_ptr(), ws.numel(), raw)
    if rc:
        _check(rc)
    return {"cache_len": new_len, "status": status}


@_on_device_of("page_table")
def cache_resize(page_table, page_refs, seqs, tokens, page_size):
    """Pages for tokens[f] tokens of sequence seqs[f] (None: f), in place: more are
    taken (lowest free number first), surplus ones released; 0 frees a sequence.

    page_table [S, max_pages] int32 (-1: no page) and page_refs [pages] int32 (0:
    free) are changed. Returns status [F]; SPEC_ENOPAGES where pages ran out
    (that sequence is left as it was).
    """
    lib = _library()
    if not page_table.is_cuda:
        raise SpecError("page_table and page_refs must be on a CUDA device")
    dev, index = page_table.device, page_table.get_device()
    S = page_table.shape[0]
    table, stride, width = _table_args(page_table, S, index)
    pages = page_refs.numel()
    refs = _owned(page_refs, (pages,), index, "page_refs")
    tok = _in(tokens, dev, index)
    who = None if seqs is None else _in(seqs, dev, index)
    if tok.dim() != 1 or (who is not None and who.shape != tok.shape):
        raise SpecError("seqs and tokens must be [F]")
    F = tok.shape[0]
    status = torch.empty((F,), dtype=torch.int32, device=dev)
    rc = lib.spec_cache_resize(table, stride, width, S, refs, pages, page_size, None if who is None else who.data_ptr(),
                               tok.data_ptr(), F, status.data_ptr(), _raw_stream(index))
    if rc:
        _check(rc)
    return {"status": status}


@_on_device_of("k_cache")
def cache_fork(k_cache, v_cache, page_table, cache_len, page_refs, src, dst):
    """Sequences dst[f] as copies of src[f], in place: full pages shared, a partly
    filled last page copied (caches [layers, pages, page_size, kv_heads, D]).

    page_table [S, max_pages], cache_len [S] and page_refs [pages] are changed;
    the dst rows must be distinct and empty. Returns status [F].
    """
    lib = _library()
    cache, sh, dt = _cache_args(k_cache, v_cache, 1)
    dev, index = k_cache.device, k_cache.get_device()
    S = page_table.shape[0]
    table, stride, width = _table_args(page_table, S, index)
    refs = _owned(page_refs, (sh[1],), index, "page_refs")
    lens = _owned(cache_len, (S,), index, "cache_len")
    a, z = _in(src, dev, index), _in(dst, dev, index)
    if a.dim() != 1 or a.shape != z.shape:
        raise SpecError("src and dst must be [F]")
    F = a.shape[0]
    status = torch.empty((F,), dtype=torch.int32, device=dev)
    raw = _raw_stream(index)
    with _turn(index, raw):
        ws = _scratch(lib.spec_cache_fork_workspace_size(F), dev, index, raw)
        rc = lib.spec_cache_fork(cache, dt, table, stride, width, S, refs, lens, a.data_ptr(), z.data_ptr(), F,
                                 status.data_ptr(), ws.data_ptr(), ws.numel(), raw)
    if rc:
        _check(rc)
    return {"status": status}


__all__ = ["use_library", "DEBUG_LIB_PATH", "philox_uniform", "verify", "verify_tree", "tree_build", "acceptance_rate", "expected_tokens",
           "walltime_factor", "ops_factor", "best_gamma", "verify_mentor", "sample", "token_logprobs", "tree_attention", "cache_append", "rotary", "Rotary",
           "cache_append_rotary", "cache_compact", "cache_weigh", "cache_evict",
           "cache_resize", "cache_fork", "load_library", "workspace",
           "SpecError", "SpecSampling", "SpecCache", "EXPORTED", "LIB_PATH"]
