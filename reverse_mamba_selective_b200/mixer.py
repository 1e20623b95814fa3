"""Thin ctypes binding of libr2l_mixer.so (include/r2l_mixer.h): argument marshalling only.

Linear attention with a decay per head (whole sequences, blocks, single tokens, gradients) and the per-head
norm of queries and keys with the rotary embedding (and its gradients).  As in ``r2l``: every step of the
computation runs in the library's CUDA kernels, on the current stream of the tensors' device unless one is given,
and there is no CPU fallback.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Dict, Optional, Tuple

import torch

from . import r2l as _r2l
from .r2l import R2L_ERR_CUDA, R2L_OK, _DTYPE_CODE, _check_dev, _ptr

MIXER_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libr2l_mixer.so")


class LinattnArgs(ctypes.Structure):
    """Mirror of r2l_linattn_args."""

    _fields_ = [
        ("batch", ctypes.c_int), ("seqlen", ctypes.c_int), ("block_len", ctypes.c_int),
        ("n_heads", ctypes.c_int), ("q_heads", ctypes.c_int), ("k_heads", ctypes.c_int), ("v_heads", ctypes.c_int),
        ("d_k", ctypes.c_int), ("d_v", ctypes.c_int),
        ("reverse", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong), ("v_stride", ctypes.c_longlong),
        ("log_decay", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
    ]


class QkNormRopeArgs(ctypes.Structure):
    """Mirror of r2l_qk_norm_rope_args."""

    _fields_ = [
        ("tokens", ctypes.c_int), ("q_heads", ctypes.c_int), ("k_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
        ("rot_dim", ctypes.c_int),
        ("interleaved", ctypes.c_int), ("position_64", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("eps", ctypes.c_float),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
        ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
        ("inv_freq", ctypes.c_void_p),
    ]


_lib = None


def load_mixer() -> ctypes.CDLL:
    """Load libr2l_mixer.so (built in-tree by reverse_mamba_selective_b200._build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(MIXER_LIB_PATH):
        raise ImportError(f"libr2l_mixer.so not found at {MIXER_LIB_PATH}; build it with "
                          "`python -m reverse_mamba_selective_b200._build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(MIXER_LIB_PATH)
    vp, ci, ll, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
    la, ro = ctypes.POINTER(LinattnArgs), ctypes.POINTER(QkNormRopeArgs)
    lib.r2l_linattn_workspace_size.argtypes = [la]
    lib.r2l_linattn_workspace_size.restype = sz
    lib.r2l_linattn.argtypes = [la, vp, vp, vp, vp, sz, vp]
    lib.r2l_linattn.restype = ci
    lib.r2l_linattn_step.argtypes = [la, vp, vp, vp, vp]
    lib.r2l_linattn_step.restype = ci
    lib.r2l_linattn_bwd_workspace_size.argtypes = [la]
    lib.r2l_linattn_bwd_workspace_size.restype = sz
    lib.r2l_linattn_bwd.argtypes = [la] + [vp] * 7 + [vp, sz, vp]
    lib.r2l_linattn_bwd.restype = ci
    lib.r2l_qk_norm_rope.argtypes = [ro, vp, ll, vp, ll, vp]
    lib.r2l_qk_norm_rope.restype = ci
    lib.r2l_qk_norm_rope_bwd_workspace_size.argtypes = [ro]
    lib.r2l_qk_norm_rope_bwd_workspace_size.restype = sz
    lib.r2l_qk_norm_rope_bwd.argtypes = [ro] + [vp] * 6 + [vp, sz, vp]
    lib.r2l_qk_norm_rope_bwd.restype = ci
    lib.r2l_mixer_device_status.argtypes = [vp]
    lib.r2l_mixer_device_status.restype = ci
    lib.r2l_mixer_last_error.argtypes = []
    lib.r2l_mixer_last_error.restype = ctypes.c_char_p
    lib.r2l_mixer_abi_version.argtypes = []
    lib.r2l_mixer_abi_version.restype = ci
    _lib = lib
    return lib


class MixerError(_r2l.R2LError):
    """A failed call of libr2l_mixer.so (``status`` as in R2LError)."""

    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {_r2l.status_string(status)}"
        if status == R2L_ERR_CUDA:
            msg += f" [{load_mixer().r2l_mixer_last_error().decode()}]"
        RuntimeError.__init__(self, msg)


def _raise(st: int, where: str):
    if st != R2L_OK:
        raise MixerError(st, where)


def _on_device(t: torch.Tensor):
    """The tensors' device made current: the library works on the current device."""
    if t.device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(t.device)


def _same_device(dev: torch.device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, not on {dev}")


def _stream_of(stream, *made):
    """The raw stream; tensors made here that another stream than the current one works on are tied to it."""
    cur = torch.cuda.current_stream().cuda_stream
    if stream is None:
        return cur
    raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if raw != cur:
        for t in made:
            if t is not None:
                t.record_stream(torch.cuda.ExternalStream(raw, device=t.device))
    return raw


def _heads(name: str, t: torch.Tensor, dtype, batch: int, seqlen: int) -> int:
    """Checks a [batch, seqlen, heads, d] operand (heads and channels dense, tokens evenly spaced) and returns its
    elements from token to token."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 4 or t.shape[0] != batch or t.shape[1] != seqlen:
        raise ValueError(f"{name} must have shape [{batch}, {seqlen}, heads, d], got {tuple(t.shape)}")
    sb, sl, sh, sd = t.stride()
    heads, d = t.shape[2], t.shape[3]
    if (d > 1 and sd != 1) or (heads > 1 and sh != d):
        raise ValueError(f"{name} must have dense heads and channels")
    tok = sl if seqlen > 1 else (sb if batch > 1 else heads * d)
    if t.numel() == 0:
        return heads * d
    if tok < heads * d or (seqlen > 1 and batch > 1 and sb != seqlen * sl):
        raise ValueError(f"{name} must have its tokens evenly spaced over batch and sequence")
    return tok


def _linattn_args(q, k, v, log_decay, scale, block_len, reverse, seq_lens) -> LinattnArgs:
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must have shape [batch, seqlen, heads, d_k]")
    dtype = q.dtype
    if dtype not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {dtype}")
    batch, seqlen = q.shape[0], q.shape[1]
    qs, ks, vs = (_heads(n, t, dtype, batch, seqlen) for n, t in (("q", q), ("k", k), ("v", v)))
    if k.shape[3] != q.shape[3]:
        raise ValueError("q and k must have the same head size")
    _check_dev("log_decay", log_decay, torch.float32)
    if log_decay.dim() != 1:
        raise ValueError("log_decay must have shape [heads]")
    _check_dev("seq_lens", seq_lens, torch.int32, (batch,))
    _same_device(q.device, k=k, v=v, log_decay=log_decay, seq_lens=seq_lens)
    d_k = q.shape[3]
    if scale is None:
        scale = d_k ** -0.5 if d_k else 1.0
    return LinattnArgs(batch, seqlen, seqlen if block_len is None else int(block_len), log_decay.shape[0], q.shape[2],
                       k.shape[2], v.shape[2], d_k, v.shape[3], int(bool(reverse)), _DTYPE_CODE[dtype], float(scale),
                       _ptr(q), _ptr(k), _ptr(v), qs, ks, vs, _ptr(log_decay), _ptr(seq_lens))


def _workspace(given: Optional[torch.Tensor], need: int, device) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], int]:
    """(workspace or None, the one made here or None, its bytes)."""
    if given is not None:
        _check_dev("workspace", given)
        _same_device(device, workspace=given)
        return given, None, given.numel() * given.element_size()
    if need == 0:
        return None, None, 0
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    return ws, ws, need


def r2l_linattn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, *,
                scale: Optional[float] = None, block_len: Optional[int] = None, reverse: bool = False,
                seq_lens: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                h_last: Optional[torch.Tensor] = None, want_h_last: bool = False, y: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with a decay per head: S_t = e^log_decay S_(t-1) + k_t v_t^T, y_t = scale q_t . S_t.

    q [b, L, q_heads, d_k], k [b, L, k_heads, d_k], v [b, L, v_heads, d_v] (bf16 or fp32; slices of a fused
    projection are fine), log_decay [heads] fp32; each head count divides ``heads``.  ``reverse`` runs right to
    left, restarting at the right edge of every ``block_len`` tokens; ``seq_lens`` [b] int32 gives the rows' own
    lengths.  h0, h_last [b, heads, d_k, d_v] fp32 (h_last may be h0).  ``scale`` defaults to d_k ** -0.5.
    Returns (y [b, L, heads, d_v], h_last or None).
    """
    lib = load_mixer()
    a = _linattn_args(q, k, v, log_decay, scale, block_len, reverse, seq_lens)
    state = (a.batch, a.n_heads, a.d_k, a.d_v)
    _check_dev("h0", h0, torch.float32, state)
    _check_dev("h_last", h_last, torch.float32, state)
    shape = (a.batch, a.seqlen, a.n_heads, a.d_v)
    _check_dev("y", y, q.dtype, shape)
    _same_device(q.device, h0=h0, h_last=h_last, y=y)
    with _on_device(q):
        made_h = made_y = None
        if h_last is None and want_h_last:
            h_last = made_h = torch.empty(state, dtype=torch.float32, device=q.device)
        if y is None:
            y = made_y = torch.empty(shape, dtype=q.dtype, device=q.device)
        ws, made, nbytes = _workspace(workspace, int(lib.r2l_linattn_workspace_size(ctypes.byref(a))), q.device)
        _raise(lib.r2l_linattn(ctypes.byref(a), _ptr(h0), _ptr(h_last), _ptr(y), _ptr(ws), nbytes,
                               _stream_of(stream, made_h, made_y, made)), "r2l_linattn")
    return y, h_last


def r2l_linattn_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, h: torch.Tensor, *,
                     scale: Optional[float] = None, h_out: Optional[torch.Tensor] = None,
                     y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of every sequence: q [b, q_heads, d_k], k [b, k_heads, d_k], v [b, v_heads, d_v], state h
    [b, heads, d_k, d_v] fp32, updated in place unless ``h_out`` is given.  Returns y [b, heads, d_v]."""
    lib = load_mixer()
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must have shape [batch, heads, d]")
    a = _linattn_args(q.unsqueeze(1), k.unsqueeze(1), v.unsqueeze(1), log_decay, scale, None, False, None)
    state = (a.batch, a.n_heads, a.d_k, a.d_v)
    if h is None:
        raise ValueError("h must be given")
    _check_dev("h", h, torch.float32, state)
    _check_dev("h_out", h_out, torch.float32, state)
    shape = (a.batch, a.n_heads, a.d_v)
    _check_dev("y", y, q.dtype, shape)
    _same_device(q.device, h=h, h_out=h_out, y=y)
    with _on_device(q):
        made = None
        if y is None:
            y = made = torch.empty(shape, dtype=q.dtype, device=q.device)
        _raise(lib.r2l_linattn_step(ctypes.byref(a), _ptr(h), _ptr(h if h_out is None else h_out), _ptr(y),
                                    _stream_of(stream, made)), "r2l_linattn_step")
    return y


def r2l_linattn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, dy: torch.Tensor, *,
                    scale: Optional[float] = None, block_len: Optional[int] = None, reverse: bool = False,
                    seq_lens: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                    dh_last: Optional[torch.Tensor] = None, want_dh0: Optional[bool] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of r2l_linattn given dy = dL/dy [b, L, heads, d_v] and dh_last = dL/dh_last (None: zero).

    Returns dq, dk, dv (the inputs' type and shapes; shared heads summed) and dh0 (fp32; by default when h0 is
    given, else None).
    """
    lib = load_mixer()
    a = _linattn_args(q, k, v, log_decay, scale, block_len, reverse, seq_lens)
    state = (a.batch, a.n_heads, a.d_k, a.d_v)
    if dy is None:
        raise ValueError("dy must be given")
    _check_dev("dy", dy, q.dtype, (a.batch, a.seqlen, a.n_heads, a.d_v))
    _check_dev("h0", h0, torch.float32, state)
    _check_dev("dh_last", dh_last, torch.float32, state)
    _same_device(q.device, dy=dy, h0=h0, dh_last=dh_last)
    if want_dh0 is None:
        want_dh0 = h0 is not None
    with _on_device(q):
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        dh0 = torch.empty(state, dtype=torch.float32, device=q.device) if want_dh0 else None
        ws, made, nbytes = _workspace(workspace, int(lib.r2l_linattn_bwd_workspace_size(ctypes.byref(a))), q.device)
        _raise(lib.r2l_linattn_bwd(ctypes.byref(a), _ptr(dy), _ptr(h0), _ptr(dh_last), _ptr(dq), _ptr(dk), _ptr(dv),
                                   _ptr(dh0), _ptr(ws), nbytes, _stream_of(stream, dq, dk, dv, dh0, made)),
               "r2l_linattn_bwd")
    return {"dq": dq, "dk": dk, "dv": dv, "dh0": dh0}


# ----------------------------------------------------------------------------- norm and rotation

def _tokens(name: str, t: torch.Tensor, dtype, tokens: int, dim: int) -> int:
    """Checks a [tokens, heads, dim] operand and returns its elements from token to token."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape[0] != tokens or t.shape[2] != dim:
        raise ValueError(f"{name} must have shape [{tokens}, heads, {dim}], got {tuple(t.shape)}")
    st, sh, sd = t.stride()
    heads = t.shape[1]
    if t.numel() == 0 or tokens == 1:
        st = heads * dim
    if (dim > 1 and sd != 1) or (heads > 1 and sh != dim) or st < heads * dim:
        raise ValueError(f"{name} must have dense heads and channels and tokens that do not overlap")
    return st


def _rope_args(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved) -> QkNormRopeArgs:
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must have shape [tokens, heads, head_dim]")
    if q.dtype not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {q.dtype}")
    tokens, _, dim = q.shape
    qs, ks = _tokens("q", q, q.dtype, tokens, dim), _tokens("k", k, q.dtype, tokens, dim)
    _check_dev("q_weight", q_weight, torch.float32, (dim,))
    _check_dev("k_weight", k_weight, torch.float32, (dim,))
    rot = 0
    if inv_freq is not None:
        _check_dev("inv_freq", inv_freq, torch.float32)
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must have shape [rot_dim / 2]")
        rot = 2 * inv_freq.shape[0]
        if positions is None:
            raise ValueError("positions must be given with inv_freq")
        if positions.dtype not in (torch.int32, torch.int64):
            raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
        _check_dev("positions", positions, None, (tokens,))
    _same_device(q.device, k=k, q_weight=q_weight, k_weight=k_weight, positions=positions, inv_freq=inv_freq)
    return QkNormRopeArgs(tokens, q.shape[1], k.shape[1], dim, rot, int(bool(interleaved)),
                          int(positions is not None and positions.dtype == torch.int64), _DTYPE_CODE[q.dtype], float(eps),
                          _ptr(q), _ptr(k), qs, ks, _ptr(q_weight), _ptr(k_weight), _ptr(positions), _ptr(inv_freq))


def r2l_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor],
                     positions: Optional[torch.Tensor], inv_freq: Optional[torch.Tensor], *, eps: float = 1e-6,
                     interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                     k_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """RMS norm of every query and key head, then the rotary embedding of its first 2 * len(inv_freq) channels.

    q [tokens, q_heads, d], k [tokens, k_heads, d] (slices of a fused projection are fine), weights [d] fp32 (None:
    ones), positions [tokens] int32 or int64, inv_freq [rot / 2] fp32 (None: no rotation).  ``interleaved`` rotates
    neighbouring channels, else channel i with i + rot / 2.  q_out may be q and k_out may be k.  Returns (q_out, k_out).
    """
    lib = load_mixer()
    a = _rope_args(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved)
    qs = _tokens("q_out", q_out, q.dtype, a.tokens, a.head_dim) if q_out is not None else 0
    ks = _tokens("k_out", k_out, q.dtype, a.tokens, a.head_dim) if k_out is not None else 0
    for name, o, t in (("q_out", q_out, q), ("k_out", k_out, k)):
        if o is not None and o.shape != t.shape:
            raise ValueError(f"{name} must have shape {tuple(t.shape)}, got {tuple(o.shape)}")
    _same_device(q.device, q_out=q_out, k_out=k_out)
    with _on_device(q):
        made_q = made_k = None
        if q_out is None:
            q_out = made_q = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k_out is None:
            k_out = made_k = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        _raise(lib.r2l_qk_norm_rope(ctypes.byref(a), _ptr(q_out), qs, _ptr(k_out), ks, _stream_of(stream, made_q, made_k)),
               "r2l_qk_norm_rope")
    return q_out, k_out


def r2l_qk_norm_rope_bwd(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor],
                         k_weight: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                         inv_freq: Optional[torch.Tensor], dq_out: torch.Tensor, dk_out: torch.Tensor, *,
                         eps: float = 1e-6, interleaved: bool = False, workspace: Optional[torch.Tensor] = None,
                         stream=None) -> Dict[str, torch.Tensor]:
    """Gradients of r2l_qk_norm_rope (q and k: its inputs) given dq_out, dk_out: dq, dk in the inputs' type and
    dq_weight, dk_weight [d] fp32 (also where the weights were None, i.e. ones)."""
    lib = load_mixer()
    a = _rope_args(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved)
    if dq_out is None or dk_out is None:
        raise ValueError("dq_out and dk_out must be given")
    _check_dev("dq_out", dq_out, q.dtype, q.shape)
    _check_dev("dk_out", dk_out, q.dtype, k.shape)
    _same_device(q.device, dq_out=dq_out, dk_out=dk_out)
    with _on_device(q):
        dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        dk = torch.empty(k.shape, dtype=q.dtype, device=q.device)
        dqw, dkw = (torch.empty(a.head_dim, dtype=torch.float32, device=q.device) for _ in range(2))
        ws, made, nbytes = _workspace(workspace, int(lib.r2l_qk_norm_rope_bwd_workspace_size(ctypes.byref(a))), q.device)
        _raise(lib.r2l_qk_norm_rope_bwd(ctypes.byref(a), _ptr(dq_out), _ptr(dk_out), _ptr(dq), _ptr(dk), _ptr(dqw), _ptr(dkw),
                                        _ptr(ws), nbytes, _stream_of(stream, dq, dk, dqw, dkw, made)),
               "r2l_qk_norm_rope_bwd")
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def r2l_mixer_device_status(stream=None) -> int:
    """Synchronise and read/clear this library's device status word (R2L_OK or R2L_ERR_TIMEOUT)."""
    return int(load_mixer().r2l_mixer_device_status(_stream_of(stream)))


def r2l_mixer_abi_version() -> int:
    return int(load_mixer().r2l_mixer_abi_version())
