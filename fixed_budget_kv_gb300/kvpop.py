"""Python binding of libkvpop (ctypes).

Argument marshalling only: every step of the hot path runs in the CUDA
library.  torch provides device memory and the current stream.  If the shared
library has not been built the import of this module still works, but every
call raises ``KvpopUnavailable`` -- there is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkvpop.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "kvpop.h")
TAU_ALL = 2147483647
LIST_QBLOCK = 64

c_int = ctypes.c_int
c_i32 = ctypes.c_int32
c_i64 = ctypes.c_int64
c_size = ctypes.c_size_t
c_float = ctypes.c_float
c_void_p = ctypes.c_void_p


class KvpopError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class KvpopUnavailable(RuntimeError):
    pass


class Budget(ctypes.Structure):
    _fields_ = [("s", c_i32), ("w", c_i32), ("k", c_i32)]


_lib = None


def header_functions() -> list[str]:
    """Names of the functions that include/kvpop.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*(kvpop_[a-z0-9_]+)\s*\(",
                                 text, flags=re.M)))


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise KvpopUnavailable(f"{path} is missing: build it with __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P = c_void_p
    sig = {
        "kvpop_status_string": ([c_int], ctypes.c_char_p),
        "kvpop_last_error": ([], ctypes.c_char_p),
        "kvpop_version": ([], c_int),
        "kvpop_device_status": ([P, c_int], c_int),
        "kvpop_mask_workspace_size": ([c_int, c_int, c_int, Budget, P], c_int),
        "kvpop_mask_lists_size": ([c_int, c_int, c_int, Budget, P], c_int),
        "kvpop_mask": ([P, c_int, c_int, c_int, Budget, P, P, P, P, P, c_size, P], c_int),
        "kvpop_attn_fwd": ([P, P, P, c_int, c_int, c_int, c_int, c_int, c_float, P, P, Budget, P, P, P],
                           c_int),
        "kvpop_attn_bwd_workspace_size": ([c_int, c_int, c_int, c_int, Budget, P], c_int),
        "kvpop_attn_bwd": ([P, P, P, P, P, P, c_int, c_int, c_int, c_int, c_int, c_float, P, P, Budget, P, P, P,
                            P, c_size, P], c_int),
        "kvpop_future_target_workspace_size": ([c_int, c_int, c_int, c_int, P], c_int),
        "kvpop_future_target": ([P, P, P, c_int, c_int, c_int, c_int, c_int, c_float, c_int, P, P, c_size,
                                 P], c_int),
        "kvpop_future_target_noalloc": ([P, P, P, c_int, c_int, c_int, c_int, c_int, c_float, c_int, P, P],
                                        c_int),
        "kvpop_target_normalize": ([P, c_int, c_int, c_int, c_int, c_int, c_float, P, P], c_int),
        "kvpop_teacher_labels": ([P, c_int, c_int, c_int, Budget, c_int, P, P, P, P], c_int),
        "kvpop_boundary_loss": ([P, P, P, P, c_int, c_int, c_int, c_int, c_int, P, c_float, P, P, P], c_int),
        "kvpop_qk_norm_rope": ([P, c_i64, P, c_i64, c_int, c_int, c_int, c_int, c_int, P, P, c_float, P, c_int, c_int, P,
                                P, P, P], c_int),
        "kvpop_qk_norm_rope_bwd_workspace_size": ([c_int, P], c_int),
        "kvpop_qk_norm_rope_bwd": ([P, c_i64, P, c_i64, P, P, c_int, c_int, c_int, c_int, c_int, P, P, c_float, P, c_int,
                                    c_int, P, P, c_i64, P, c_i64, P, P, P, c_size, P], c_int),
        "kvpop_prefix_attn_workspace_size": ([c_int, c_int, c_int, c_int, c_int, c_int, P], c_int),
        "kvpop_prefix_attn": ([P, P, P, c_int, c_int, c_int, c_int, c_int, c_int, c_float, P, P, P, P, P, P, P, c_size,
                               P], c_int),
        "kvpop_paged_append": ([P, c_i64, P, c_i64, c_int, c_int, c_int, c_int, P, P, P, c_int, P, c_i64, P, c_i64, c_int,
                                c_int, P, P], c_int),
        "kvpop_paged_attn_workspace_size": ([c_int] * 7 + [P], c_int),
        "kvpop_paged_attn": ([P, c_int, c_int, c_int, c_int, c_int, c_float, P, P, P, c_int, P, c_i64, P, c_i64, c_int, c_int,
                              P, P, P, c_size, P], c_int),
        "kvpop_paged_mass_workspace_size": ([c_int] * 7 + [P], c_int),
        "kvpop_paged_mass": ([P, P, c_int, c_int, c_int, c_int, c_int, c_float, c_float, P, P, P, c_int, P, c_i64, c_int,
                              c_int, P, P, c_size, P], c_int),
        "kvpop_paged_evict": ([P, c_i64, P, c_i64, P, c_int, c_int, c_int, Budget, P, P, c_int, c_int, c_int, P, P, P],
                              c_int),
        "kvpop_cache_create": ([c_int, c_int, c_int, c_int, Budget, P], c_int),
        "kvpop_cache_destroy": ([P], c_int),
        "kvpop_cache_prefill": ([P, P, P, P, c_int, P, P], c_int),
        "kvpop_decode_step": ([P, P, P, P, P, P, P, P, P], c_int),
        "kvpop_cache_slots": ([P, P, P], c_int),
        "kvpop_cache_position": ([P, P], c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def available() -> bool:
    try:
        load()
        return True
    except (KvpopUnavailable, OSError):
        return False


def _check(st: int, what: str):
    if st != 0:
        lib = load()
        msg = lib.kvpop_status_string(st).decode()
        detail = lib.kvpop_last_error().decode()
        raise KvpopError(st, f"{what}: {msg}: {detail}")


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    if stream is None:  # the handle itself: building a torch.cuda.Stream costs several microseconds a call
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _need(t, dtype, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _device(t, name):
    """Index of the CUDA device that t is on, which has to be the current one."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}: make it the current device first")
    return dev


def _fit(t, dtype, dev, shape, name):
    """A contiguous CUDA tensor of this type and shape on device dev."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return
    _need(t, dtype, name)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


_here = contextlib.nullcontext()


def _empty_as(t):
    # torch.empty alone: every further torch function next to a launch costs the host about a microsecond
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _on(stream):
    """Memory that a call allocates belongs to the stream that uses it."""
    return _here if stream is None else torch.cuda.stream(stream)


def device_status(reset: bool = True):
    out = (c_i32 * 4)()
    st = load().kvpop_device_status(ctypes.cast(out, c_void_p), int(reset))
    return st, list(out)


# ----------------------------------------------------------------------------
# mask
# ----------------------------------------------------------------------------

def mask_workspace_size(b, H, S, s, w, k) -> int:
    n = c_size()
    _check(load().kvpop_mask_workspace_size(b, H, S, Budget(s, w, k), ctypes.byref(n)), "mask_workspace_size")
    return n.value


def mask_lists_size(b, H, S, s, w, k) -> int:
    n = c_size()
    _check(load().kvpop_mask_lists_size(b, H, S, Budget(s, w, k), ctypes.byref(n)), "mask_lists_size")
    return n.value


def mask(prio: torch.Tensor, s: int, w: int, k: int, lists: bool = True, workspace=None, out=None,
         stream=None):
    """rank, tau, evict_at [b,H,S] int32 and the long-range lists [b,H,ceil(S/64),k,2]
    (position, evict_at) for priorities [b,H,S] fp32."""
    _need(prio, torch.float32, "prio")
    b, H, S = prio.shape
    lib = load()
    dev = prio.device
    if out is None:
        rank = torch.empty((b, H, S), dtype=torch.int32, device=dev)
        tau = torch.empty_like(rank)
        ev = torch.empty_like(rank)
        nl = (S + LIST_QBLOCK - 1) // LIST_QBLOCK
        lst = torch.empty((b, H, nl, max(k, 0), 2), dtype=torch.int32, device=dev) if (lists and k > 0) else None
    else:
        rank, tau, ev, lst = out
    if workspace is None:
        workspace = torch.empty(mask_workspace_size(b, H, S, s, w, k), dtype=torch.uint8, device=dev)
    _check(lib.kvpop_mask(_p(prio), b, H, S, Budget(s, w, k), _p(rank), _p(tau), _p(ev), _p(lst),
                          _p(workspace), workspace.numel(), _stream(stream)), "kvpop_mask")
    return rank, tau, ev, lst


# ----------------------------------------------------------------------------
# attention and target
# ----------------------------------------------------------------------------

def attn_fwd(q, k, v, scale: float = 0.0, evict_at=None, lists=None, budget=(0, 0, 0), want_o=True,
             out=None, stream=None):
    """Sparse (evict_at/lists given) or dense causal attention.  Returns (O or None, lse)."""
    _need(q, torch.bfloat16, "q")
    _need(k, torch.bfloat16, "k")
    if v is not None:
        _need(v, torch.bfloat16, "v")
    b, S, Hq, D = q.shape
    H = k.shape[2]
    if out is None:
        O = torch.empty_like(q) if want_o else None
        lse = torch.empty((b, Hq, S), dtype=torch.float32, device=q.device)
    else:
        O, lse = out
    _check(load().kvpop_attn_fwd(_p(q), _p(k), _p(v), b, S, Hq, H, D, float(scale), _p(evict_at),
                                 _p(lists), Budget(*budget), _p(O), _p(lse), _stream(stream)),
           "kvpop_attn_fwd")
    return O, lse


def attn_bwd_workspace_size(b, S, Hq, H, budget) -> int:
    n = c_size()
    _check(load().kvpop_attn_bwd_workspace_size(b, S, Hq, H, Budget(*budget), ctypes.byref(n)),
           "attn_bwd_workspace_size")
    return n.value


def attn_bwd(q, k, v, O, dO, lse, evict_at, lists, budget, scale: float = 0.0, workspace=None, out=None,
             stream=None):
    """Gradient of the sparse attention: (dq [b,S,Hq,D], dk, dv [b,S,H,D]), fp32.

    O and lse are the forward's outputs for the same inputs; dO is the upstream
    gradient (bf16, the shape of q)."""
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (O, "O"), (dO, "dO")):
        _need(t, torch.bfloat16, name)
    _need(lse, torch.float32, "lse")
    b, S, Hq, D = q.shape
    H = k.shape[2]
    if workspace is None:
        workspace = torch.empty(attn_bwd_workspace_size(b, S, Hq, H, budget), dtype=torch.uint8, device=q.device)
    if out is None:
        dq = torch.empty((b, S, Hq, D), dtype=torch.float32, device=q.device)
        dk = torch.empty((b, S, H, D), dtype=torch.float32, device=q.device)
        dv = torch.empty_like(dk)
    else:
        dq, dk, dv = out
    _check(load().kvpop_attn_bwd(_p(q), _p(k), _p(v), _p(O), _p(dO), _p(lse), b, S, Hq, H, D, float(scale),
                                 _p(evict_at), _p(lists), Budget(*budget), _p(dq), _p(dk), _p(dv), _p(workspace),
                                 workspace.numel(), _stream(stream)), "kvpop_attn_bwd")
    return dq, dk, dv


def target_workspace_size(b, S, Hq, H) -> int:
    n = c_size()
    _check(load().kvpop_future_target_workspace_size(b, S, Hq, H, ctypes.byref(n)),
           "future_target_workspace_size")
    return n.value


def future_target(q, k, lse, w: int, scale: float = 0.0, workspace=None, out=None, stream=None):
    """log future-attention mass per (batch, KV head, token): [b,H,S] fp32."""
    _need(q, torch.bfloat16, "q")
    _need(k, torch.bfloat16, "k")
    _need(lse, torch.float32, "lse")
    b, S, Hq, D = q.shape
    H = k.shape[2]
    if workspace is None:
        workspace = torch.empty(target_workspace_size(b, S, Hq, H), dtype=torch.uint8, device=q.device)
    target = torch.empty((b, H, S), dtype=torch.float32, device=q.device) if out is None else out
    _check(load().kvpop_future_target(_p(q), _p(k), _p(lse), b, S, Hq, H, D, float(scale), int(w),
                                      _p(target), _p(workspace), workspace.numel(), _stream(stream)),
           "kvpop_future_target")
    return target


def future_target_noalloc(q, k, lse, w: int, scale: float = 0.0, out=None, stream=None):
    """Same result as future_target, for callers that cannot allocate device
    memory: the pass's scratch lives in a fixed 16 MiB array inside the library
    (problems needing more raise KvpopError).  Only the output is allocated here,
    and only when `out` is not given."""
    _need(q, torch.bfloat16, "q")
    _need(k, torch.bfloat16, "k")
    _need(lse, torch.float32, "lse")
    b, S, Hq, D = q.shape
    H = k.shape[2]
    target = torch.empty((b, H, S), dtype=torch.float32, device=q.device) if out is None else out
    _check(load().kvpop_future_target_noalloc(_p(q), _p(k), _p(lse), b, S, Hq, H, D, float(scale), int(w),
                                              _p(target), _stream(stream)), "kvpop_future_target_noalloc")
    return target


# ----------------------------------------------------------------------------
# training-side passes: normalised target, teacher labels, boundary loss
# ----------------------------------------------------------------------------

def target_normalize(target, G: int, w: int, eps: float, out=None, stream=None):
    """r_tgt = log(eps + exp(target) / (G * N_t)), N_t = S - t - w, [b, H, S]."""
    _need(target, torch.float32, "target")
    b, H, S = target.shape
    r = torch.empty_like(target) if out is None else out
    _check(load().kvpop_target_normalize(_p(target), b, H, S, int(G), int(w), float(eps), _p(r), _stream(stream)),
           "kvpop_target_normalize")
    return r


def teacher_labels(r_tgt, s: int, w: int, k: int, n: int, log_gamma, out=None, stream=None):
    """(t_bnd, y) per row, int32 [b, H, S]; log_gamma: fp32 [H] on the device."""
    _need(r_tgt, torch.float32, "r_tgt")
    _need(log_gamma, torch.float32, "log_gamma")
    b, H, S = r_tgt.shape
    if out is None:
        tb = torch.empty((b, H, S), dtype=torch.int32, device=r_tgt.device)
        y = torch.empty_like(tb)
    else:
        tb, y = out
    _check(load().kvpop_teacher_labels(_p(r_tgt), b, H, S, Budget(s, w, k), int(n), _p(log_gamma), _p(tb), _p(y),
                                       _stream(stream)), "kvpop_teacher_labels")
    return tb, y


def boundary_loss(r_hat, t_bnd, y, w: int, n: int, log_gamma, tau: float, omega=None, out=None, stream=None):
    """(loss[2] = (mean loss, pair count), grad [b, H, S]) of the pairwise boundary loss."""
    _need(r_hat, torch.float32, "r_hat")
    b, H, S = r_hat.shape
    if out is None:
        loss = torch.empty(2, dtype=torch.float32, device=r_hat.device)
        grad = torch.empty_like(r_hat)
    else:
        loss, grad = out
    _check(load().kvpop_boundary_loss(_p(r_hat), _p(t_bnd), _p(y), _p(omega), b, H, S, int(w), int(n),
                                      _p(log_gamma), float(tau), _p(loss), _p(grad), _stream(stream)),
           "kvpop_boundary_loss")
    return loss, grad


# ----------------------------------------------------------------------------
# before the attention: per-head norm of q and k with the position rotation
# ----------------------------------------------------------------------------

def _token_stride(t, shape, dev, name):
    """Elements between the tokens of a bf16 [b, S, heads, D] view whose heads are contiguous."""
    if t.dtype is not torch.bfloat16 or t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype is not torch.bfloat16:
            raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    b, S, heads, D = shape
    if t.is_contiguous():
        return heads * D
    s0, s1, s2, s3 = t.stride()
    if s3 != 1 or (heads > 1 and s2 != D):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if S > 1:
        if b > 1 and s0 != S * s1:
            raise ValueError(f"{name}: the tokens must be evenly spaced over the batch")
        return s1
    return s0 if b > 1 else heads * D


def _qk_args(q, k, wq, wk, inv_freq, pos):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [b, S, Hq, D] and k [b, S, H, D]")
    b, S, Hq, D = q.shape
    H = k.shape[2]
    dev = _device(q, "q")
    sq, sk = _token_stride(q, (b, S, Hq, D), dev, "q"), _token_stride(k, (b, S, H, D), dev, "k")
    if wq is not None:
        _fit(wq, torch.float32, dev, (D,), "wq")
    if wk is not None:
        _fit(wk, torch.float32, dev, (D,), "wk")
    R = 0
    if inv_freq is not None:
        R = 2 * inv_freq.numel()
        _fit(inv_freq, torch.float32, dev, (R // 2,), "inv_freq")
    if pos is not None:
        _fit(pos, torch.int32, dev, (b, S), "pos")
    return dev, sq, sk, b, S, Hq, H, D, R


def qk_norm_rope(q, k, wq, wk, eps: float, inv_freq, pos=None, interleaved: bool = False, out=None, stream=None):
    """RMS norm of each head of q [b,S,Hq,D] and k [b,S,H,D] (weights wq, wk: fp32 [D] or
    None) and the rotation of the first 2 * len(inv_freq) dims at positions pos (int32
    [b,S]; None: 0..S-1).  q and k may be views of a packed projection.  Returns
    contiguous (q_out, k_out); a decode step's n tokens are [n,1,heads,D]."""
    dev, sq, sk, b, S, Hq, H, D, R = _qk_args(q, k, wq, wk, inv_freq, pos)
    if out is None:
        with _on(stream):
            qo, ko = _empty_as(q), _empty_as(k)
    else:
        qo, ko = out
        _fit(qo, torch.bfloat16, dev, q.shape, "q_out")
        _fit(ko, torch.bfloat16, dev, k.shape, "k_out")
    st = load().kvpop_qk_norm_rope(_p(q), sq, _p(k), sk, b, S, Hq, H, D, _p(wq), _p(wk), eps, _p(inv_freq), R,
                                   1 if interleaved else 0, _p(pos), _p(qo), _p(ko), _stream(stream))
    if st:
        _check(st, "kvpop_qk_norm_rope")
    return qo, ko


@functools.lru_cache(maxsize=None)
def qk_norm_rope_bwd_workspace_size(D: int) -> int:
    n = c_size()
    _check(load().kvpop_qk_norm_rope_bwd_workspace_size(D, ctypes.byref(n)), "qk_norm_rope_bwd_workspace_size")
    return n.value


def qk_norm_rope_bwd(q, k, dq, dk, wq, wk, eps: float, inv_freq, pos=None, interleaved: bool = False, workspace=None,
                     out=None, stream=None):
    """Gradient of qk_norm_rope for the upstream fp32 dq [b,S,Hq,D] and dk [b,S,H,D]
    (attn_bwd's): (dq_in, dk_in bf16, dwq, dwk fp32 [D]).  q and k are the forward's
    inputs.  `out` may hold views of a packed projection's gradient, and None for a
    weight gradient that is not wanted."""
    dev, sq, sk, b, S, Hq, H, D, R = _qk_args(q, k, wq, wk, inv_freq, pos)
    _fit(dq, torch.float32, dev, q.shape, "dq")
    _fit(dk, torch.float32, dev, k.shape, "dk")
    with _on(stream):
        if workspace is None:
            workspace = torch.empty(qk_norm_rope_bwd_workspace_size(D), dtype=torch.uint8, device=q.device)
        else:
            _fit(workspace, torch.uint8, dev, workspace.shape, "workspace")
        if out is None:
            dqi, dki = _empty_as(q), _empty_as(k)
            dwq, dwk = (torch.empty(D, dtype=torch.float32, device=q.device) for _ in range(2))
            so, sp = Hq * D, H * D
        else:
            dqi, dki, dwq, dwk = out
            so, sp = _token_stride(dqi, q.shape, dev, "dq_in"), _token_stride(dki, k.shape, dev, "dk_in")
            if dwq is not None:
                _fit(dwq, torch.float32, dev, (D,), "dwq")
            if dwk is not None:
                _fit(dwk, torch.float32, dev, (D,), "dwk")
    _check(load().kvpop_qk_norm_rope_bwd(_p(q), sq, _p(k), sk, _p(dq), _p(dk), b, S, Hq, H, D, _p(wq), _p(wk), eps,
                                         _p(inv_freq), R, 1 if interleaved else 0, _p(pos), _p(dqi), so, _p(dki), sp,
                                         _p(dwq), _p(dwk), _p(workspace), workspace.numel(), _stream(stream)),
           "kvpop_qk_norm_rope_bwd")
    return dqi, dki, dwq, dwk


# ----------------------------------------------------------------------------
# decode over shared prefixes
# ----------------------------------------------------------------------------

def prefix_attn_workspace_size(n, m, P, Hq, H, D) -> int:
    return _prefix_workspace(torch.cuda.current_device() if torch.cuda.is_available() else -1, n, m, P, Hq, H, D)


@functools.lru_cache(maxsize=1024)
def _prefix_workspace(dev, n, m, P, Hq, H, D) -> int:
    """Bytes on device dev: a function of the sizes and of the device's number of SMs."""
    nb = c_size()
    _check(load().kvpop_prefix_attn_workspace_size(n, m, P, Hq, H, D, ctypes.byref(nb)), "prefix_attn_workspace_size")
    return nb.value


def prefix_attn(q, pk, pv, cu=None, lens=None, join=None, scale: float = 0.0, workspace=None, out=None, stream=None):
    """Attention of decode rows q [n,Hq,D] over prefixes pk, pv [m,P,H,D] that groups of
    sequences share: group j is the sequences cu[j]..cu[j+1]-1 (int32 [m+1]; None with
    one prefix) and sees the first lens[j] keys (int32 [m]; None: all P).  `join` =
    (O2 [n,Hq,D] bf16, lse2 [n,Hq] fp32), the rows' attention over other keys such as
    Cache.step's, makes the result the attention over both.  Returns (O, lse), [n,Hq,D]
    bf16 and [n,Hq] fp32; rows outside the groups are not written."""
    if q.dim() != 3 or pk.dim() != 4:
        raise ValueError("q must be [n, Hq, D] and pk [m, P, H, D]")
    n, Hq, D = rows = q.shape
    m, P, H, _ = pk.shape
    dev = _device(q, "q")
    _fit(q, torch.bfloat16, dev, rows, "q")
    _fit(pk, torch.bfloat16, dev, (m, P, H, D), "pk")
    _fit(pv, torch.bfloat16, dev, (m, P, H, D), "pv")
    if cu is not None:
        _fit(cu, torch.int32, dev, (m + 1,), "cu")
    if lens is not None:
        _fit(lens, torch.int32, dev, (m,), "lens")
    O2 = lse2 = None
    if join is not None:
        O2, lse2 = join
        _fit(O2, torch.bfloat16, dev, rows, "O2")
        _fit(lse2, torch.float32, dev, (n, Hq), "lse2")
    with _on(stream):
        if out is None:
            O, lse = _empty_as(q), torch.empty((n, Hq), dtype=torch.float32, device=q.device)
        else:
            O, lse = out
            _fit(O, torch.bfloat16, dev, rows, "O")
            _fit(lse, torch.float32, dev, (n, Hq), "lse")
        if workspace is None:
            workspace = torch.empty(_prefix_workspace(dev, n, m, P, Hq, H, D), dtype=torch.uint8, device=q.device)
        else:
            _fit(workspace, torch.uint8, dev, workspace.shape, "workspace")
    _check(load().kvpop_prefix_attn(_p(q), _p(pk), _p(pv), n, m, P, Hq, H, D, scale, _p(cu), _p(lens), _p(O2),
                                    _p(lse2), _p(O), _p(lse), _p(workspace), workspace.numel(), _stream(stream)),
           "kvpop_prefix_attn")
    return O, lse


# ----------------------------------------------------------------------------
# paged cache
# ----------------------------------------------------------------------------

def _page_stride(x, dev, name):
    """Elements between the pages of a bf16 [pages, H, page, D] cache whose pages are contiguous."""
    if x.is_contiguous() and x.dtype is torch.bfloat16 and x.get_device() == dev:
        return x.stride(0) if x.shape[0] > 1 else x.numel()  # of one page it means nothing
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {x.dtype}")
    if x.get_device() != dev:
        raise ValueError(f"{name} is on {x.device}, not on cuda:{dev}")
    if not x[:1].is_contiguous():
        raise ValueError(f"{name}: a page must be contiguous")
    pages, H, page, D = x.shape
    return x.stride(0) if pages > 1 else H * page * D


def _row_stride(t, T, H, D, dev, name):
    """Elements between the tokens of a bf16 [T, H, D] view whose heads are contiguous."""
    if t.dtype is torch.bfloat16 and t.get_device() == dev and t.shape == (T, H, D):
        if t.is_contiguous():
            return H * D
        s0, s1, s2 = t.stride()
        if s2 == 1 and (s1 == D or H == 1):
            return s0 if T > 1 else H * D
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return _token_stride(t[:, None], (T, 1, H, D), dev, name)


def _paged_args(kp, vp, table, lens, cu, T, D, dev):
    """(pages, H, page, elements between the pages of kp and of vp, n, max_pages) of a call with T
    rows; vp may be None."""
    shape = kp.shape
    if len(shape) != 4 or shape[3] != D:
        raise ValueError(f"kp must be [pages, H, page, {D}], got {list(shape)}")
    if table.dim() != 2:
        raise ValueError("table must be [n, max_pages]")
    n, most = table.shape
    i32 = torch.int32
    # the cheap questions together: a small call costs the host more than the GPU
    if not (table.dtype is i32 and lens.dtype is i32 and table.get_device() == dev and lens.get_device() == dev
            and table.is_contiguous() and lens.is_contiguous() and lens.shape == (n,)):
        _fit(table, i32, dev, (n, most), "table")
        _fit(lens, i32, dev, (n,), "lens")
    if cu is not None:
        _fit(cu, i32, dev, (n + 1,), "cu")
    elif T != n:
        raise ValueError(f"cu is needed with {T} rows of {n} sequences")
    pk = _page_stride(kp, dev, "kp")
    if vp is None:
        return shape[0], shape[1], shape[2], pk, 0, n, most
    if vp.shape != shape:
        raise ValueError(f"vp must be {list(shape)}, got {list(vp.shape)}")
    return shape[0], shape[1], shape[2], pk, _page_stride(vp, dev, "vp"), n, most


def paged_append(k_new, v_new, kp, vp, table, lens, cu=None, scores=None, stream=None):
    """New tokens' k_new, v_new [T,H,D] (views of a packed projection, too) into the pages
    kp, vp [pages,H,page,D]: rows cu[i]..cu[i+1]-1 (int32 [n+1]; None: one each) become the
    last of the lens[i] slots that table [n,max_pages] gives sequence i.  The weights of
    the new slots in scores [pages,H,page] become 0."""
    if k_new.dim() != 3:
        raise ValueError("k_new must be [T, H, D]")
    T, H, D = k_new.shape
    dev = _device(k_new, "k_new")
    sk, sv = _row_stride(k_new, T, H, D, dev, "k_new"), _row_stride(v_new, T, H, D, dev, "v_new")
    pages, heads, page, pk, pv, n, most = _paged_args(kp, vp, table, lens, cu, T, D, dev)
    if heads != H:
        raise ValueError(f"kp must be [pages, {H}, page, {D}], got {list(kp.shape)}")
    if scores is not None:
        _fit(scores, torch.float32, dev, (pages, H, page), "scores")
    st = load().kvpop_paged_append(_p(k_new), sk, _p(v_new), sv, T, n, H, D, _p(cu), _p(lens), _p(table), most, _p(kp), pk,
                                   _p(vp), pv, pages, page, _p(scores), _stream(stream))
    if st:
        _check(st, "kvpop_paged_append")


@functools.lru_cache(maxsize=1024)
def _paged_workspace(what, dev, T, n, Hq, H, D, most, page) -> int:
    """Bytes on device dev: a function of the sizes and of the device's number of SMs."""
    nb = c_size()
    name = f"kvpop_paged_{what}_workspace_size"
    _check(getattr(load(), name)(T, n, Hq, H, D, most, page, ctypes.byref(nb)), name)
    return nb.value


def _paged_scratch(what, workspace, dev, T, n, Hq, H, D, most, page, handle):
    """Address and bytes of the caller's workspace, or of one for this call, which goes back by
    _scratch_back: plain memory of torch's allocator, taken and given in the order of the stream (the
    first tensor that a call makes next to a launch costs the host 5 us, plain memory half a one)."""
    if workspace is None:
        nb = _paged_workspace(what, dev, T, n, Hq, H, D, most, page)
        return torch._C._cuda_cudaCachingAllocator_raw_alloc(nb, handle), nb
    _fit(workspace, torch.uint8, dev, workspace.shape, "workspace")
    return workspace.data_ptr(), workspace.numel()


def _scratch_back(workspace, ws):
    if workspace is None:
        torch._C._cuda_cudaCachingAllocator_raw_delete(ws)


def paged_attn_workspace_size(T, n, Hq, H, D, max_pages, page) -> int:
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    return _paged_workspace("attn", dev, T, n, Hq, H, D, max_pages, page)


def paged_mass_workspace_size(T, n, Hq, H, D, max_pages, page) -> int:
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    return _paged_workspace("mass", dev, T, n, Hq, H, D, max_pages, page)


def paged_attn(q, kp, vp, table, lens, cu=None, scale: float = 0.0, workspace=None, out=None, stream=None):
    """Causal attention of new tokens q [T,Hq,D] over the slots that their sequences hold,
    their own among them (appended before): table, lens, cu as for paged_append.  Returns
    (O [T,Hq,D] bf16, lse [T,Hq] fp32); rows of no sequence are not written."""
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, D]")
    T, Hq, D = rows = q.shape
    dev = _device(q, "q")
    _fit(q, torch.bfloat16, dev, rows, "q")
    pages, H, page, pk, pv, n, most = _paged_args(kp, vp, table, lens, cu, T, D, dev)
    if out is not None:
        O, lse = out
        _fit(O, torch.bfloat16, dev, rows, "O")
        _fit(lse, torch.float32, dev, (T, Hq), "lse")
    elif stream is None:
        O, lse = torch.empty_like(q), torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    else:
        with _on(stream):
            O, lse = torch.empty_like(q), torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    s = _stream(stream)
    ws, nb = _paged_scratch("attn", workspace, dev, T, n, Hq, H, D, most, page, s)
    try:
        st = load().kvpop_paged_attn(_p(q), T, n, Hq, H, D, scale, _p(cu), _p(lens), _p(table), most, _p(kp), pk, _p(vp), pv,
                                     pages, page, _p(O), _p(lse), ws, nb, s)
    finally:
        _scratch_back(workspace, ws)
    if st:
        _check(st, "kvpop_paged_attn")
    return O, lse


def paged_mass(q, lse, kp, scores, table, lens, cu=None, scale: float = 0.0, decay: float = 1.0, workspace=None,
               stream=None):
    """scores [pages,H,page] fp32 = decay * scores + the attention weight that each held key
    receives from the rows of q [T,Hq,D], whose log-sum-exp lse [T,Hq] is paged_attn's.  The
    rows may be the last ones of each chunk only (an observation window).  Returns scores."""
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, D]")
    T, Hq, D = rows = q.shape
    dev = _device(q, "q")
    _fit(q, torch.bfloat16, dev, rows, "q")
    _fit(lse, torch.float32, dev, (T, Hq), "lse")
    pages, H, page, pk, _, n, most = _paged_args(kp, None, table, lens, cu, T, D, dev)
    _fit(scores, torch.float32, dev, (pages, H, page), "scores")
    s = _stream(stream)
    ws, nb = _paged_scratch("mass", workspace, dev, T, n, Hq, H, D, most, page, s)
    try:
        st = load().kvpop_paged_mass(_p(q), _p(lse), T, n, Hq, H, D, scale, decay, _p(cu), _p(lens), _p(table), most, _p(kp),
                                     pk, pages, page, _p(scores), ws, nb, s)
    finally:
        _scratch_back(workspace, ws)
    if st:
        _check(st, "kvpop_paged_mass")
    return scores


def paged_evict(kp, vp, scores, table, lens, s: int, w: int, k: int, out=None, stream=None):
    """Each head of the sequences with more than B = s + w + k slots keeps its first s, its
    last w and the k of the others with the highest scores, moved to slots 0..B-1 in their
    order.  Returns (kept [n,H,B] int32: the old slot of each new one, -1 behind the new
    length; new_lens [n] int32)."""
    if kp.dim() != 4:
        raise ValueError("kp must be [pages, H, page, D]")
    D, dev = kp.shape[3], _device(kp, "kp")
    pages, H, page, pk, pv, n, most = _paged_args(kp, vp, table, lens, None, table.shape[0], D, dev)
    _fit(scores, torch.float32, dev, (pages, H, page), "scores")
    B = s + w + k
    if out is None:
        with _on(stream):
            kept = torch.empty((n, H, max(B, 0)), dtype=torch.int32, device=kp.device)
            new = torch.empty(n, dtype=torch.int32, device=kp.device)
    else:
        kept, new = out
        _fit(kept, torch.int32, dev, (n, H, B), "kept")
        _fit(new, torch.int32, dev, (n,), "new_lens")
    st = load().kvpop_paged_evict(_p(kp), pk, _p(vp), pv, _p(scores), n, H, D, Budget(s, w, k), _p(lens), _p(table), most,
                                  pages, page, _p(kept), _p(new), _stream(stream))
    if st:
        _check(st, "kvpop_paged_evict")
    return kept, new


# ----------------------------------------------------------------------------
# decode
# ----------------------------------------------------------------------------

class Cache:
    """Fixed-budget decode cache of B = s + w + k slots per (sequence, KV head)."""

    def __init__(self, n: int, H: int, G: int, D: int, s: int, w: int, k: int):
        self.n, self.H, self.G, self.D = n, H, G, D
        self.s, self.w, self.k = s, w, k
        self.B = s + w + k
        self._h = c_void_p()
        _check(load().kvpop_cache_create(n, H, G, D, Budget(s, w, k), ctypes.byref(self._h)),
               "kvpop_cache_create")

    def close(self):
        if self._h:
            load().kvpop_cache_destroy(self._h)
            self._h = c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prefill(self, k, v, prio, evict_at, stream=None):
        _need(k, torch.bfloat16, "k")
        _need(v, torch.bfloat16, "v")
        _need(prio, torch.float32, "prio")
        _need(evict_at, torch.int32, "evict_at")
        P = k.shape[1]
        _check(load().kvpop_cache_prefill(self._h, _p(k), _p(v), _p(prio), P, _p(evict_at), _stream(stream)),
               "kvpop_cache_prefill")

    def step(self, q_new, k_new, v_new, prio_new, out=None, stream=None):
        if out is None:
            O = torch.empty_like(q_new)
            lse = torch.empty(q_new.shape[:2], dtype=torch.float32, device=q_new.device)
            ev = torch.empty((self.n, self.H), dtype=torch.int32, device=q_new.device)
        else:
            O, lse, ev = out
        _check(load().kvpop_decode_step(self._h, _p(q_new), _p(k_new), _p(v_new), _p(prio_new), _p(O),
                                        _p(lse), _p(ev), _stream(stream)), "kvpop_decode_step")
        return O, lse, ev

    def slots(self, stream=None):
        out = torch.empty((self.n, self.H, self.B), dtype=torch.int32, device="cuda")
        _check(load().kvpop_cache_slots(self._h, _p(out), _stream(stream)), "kvpop_cache_slots")
        return out

    def position(self) -> int:
        q = c_i32()
        _check(load().kvpop_cache_position(self._h, ctypes.byref(q)), "kvpop_cache_position")
        return q.value
