"""Thin ctypes binding of libr2l_mixer.so (include/r2l_mixer.h): argument marshalling only.

Linear attention with a decay per head (whole sequences, blocks, single tokens, gradients) and the per-head
norm of queries and keys with the rotary embedding (and its gradients).  As in ``r2l``: every step of the
computation runs in the library's CUDA kernels, on the current stream of the tensors' device unless one is given,
and there is no CPU fallback.  Outputs and workspaces that a call makes come from the memory of the stream it works on;
inputs that were made on another one have to be ready there, and stay until the call is done, as for any torch operator.
"""

from __future__ import annotations

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


class _Place:
    """Where a call works: makes the tensors' device current (the library works on the current device), and the given
    stream, so that what is allocated in here comes from that stream's memory: a block that another stream has freed may
    still be in use there.  Entering gives the raw stream."""

    __slots__ = ("raw", "caller", "inner")

    def __init__(self, stream, index: int):
        self.raw = torch._C._cuda_getCurrentRawStream(index)
        self.caller = self.inner = None
        if stream is not None:
            raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
            if raw != self.raw:
                self.raw, self.caller = raw, torch.cuda.current_stream(index)
                self.inner = torch.cuda.stream(torch.cuda.ExternalStream(raw, device=index))
                return
        if index != torch._C._cuda_getDevice():
            self.inner = torch.cuda.device(index)

    def __enter__(self) -> int:
        if self.inner is not None:
            self.inner.__enter__()
        return self.raw

    def __exit__(self, *exc):
        if self.inner is not None:
            self.inner.__exit__(*exc)
        return False

    def give(self, *made):
        """Ties outputs that were made for another stream to the caller's as well, where they are used next."""
        if self.caller is not None:
            for t in made:
                if t is not None:
                    t.record_stream(self.caller)


def _ptr_of(name: str, t: Optional[torch.Tensor], dtype, shape, index: int) -> Optional[int]:
    """The address of an optional dense tensor of the given type, shape (None: any) and device."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or not t.is_contiguous() or (shape is not None and t.shape != shape):
        _check_dev(name, t, dtype, shape)  # says what is wrong
    if t.get_device() != index:
        raise (ValueError if t.is_cuda else TypeError)(f"{name} must be on cuda:{index}, got {t.device}")
    return t.data_ptr()


def _first(name: str, t, dims: int) -> int:
    """The CUDA device of the first operand, which has to have a supported type and ``dims`` dimensions."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(t.shape)}")
    if t.dtype not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return t.get_device()


def _heads(name: str, t: torch.Tensor, dtype, lead: Tuple[int, ...], index: int) -> int:
    """Checks a [*lead, heads, d] operand (heads and channels dense, tokens evenly spaced over lead) and returns its
    elements from token to token (0: dense)."""
    shape = t.shape if isinstance(t, torch.Tensor) else ()
    fits = len(shape) == len(lead) + 2 and shape[:-2] == lead
    if fits and t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        return 0
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not fits:
        raise ValueError(f"{name} must have shape [{', '.join(map(str, lead))}, heads, d], got {tuple(shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    strides = t.stride()
    heads, d = shape[-2], shape[-1]
    if (d > 1 and strides[-1] != 1) or (heads > 1 and strides[-2] != d):
        raise ValueError(f"{name} must have dense heads and channels")
    # the innermost dimension of lead that has more than one entry gives the tokens' distance (none has: dense), the others
    # follow from it; a distance of 0 is a broadcast, whose tokens the library would read as dense
    tok = want = None
    for n, st in zip(reversed(lead), reversed(strides[:-2])):
        if n == 1:
            continue
        if tok is None:
            if st < heads * d:
                raise ValueError(f"{name} must not have overlapping tokens")
            tok = want = st
        elif st != want:
            raise ValueError(f"{name} must have its tokens evenly spaced")
        want *= n
    return tok or 0


def _int32(what: str, *sizes: int):
    """Sizes that the C structures hold in 32 bits: ctypes would cut a longer one off in silence."""
    if max(sizes) > 0x7FFFFFFF or min(sizes) < -0x80000000:
        raise ValueError(f"{what} must be below 2^31, got {sizes}")


def _linattn_args(q, k, v, log_decay, scale, block_len, reverse, seq_lens, lead, index) -> LinattnArgs:
    dtype = q.dtype
    qs, ks, vs = _heads("q", q, dtype, lead, index), _heads("k", k, dtype, lead, index), _heads("v", v, dtype, lead, index)
    batch, seqlen = lead if len(lead) == 2 else (lead[0], 1)
    q_heads, d_k = q.shape[-2:]
    k_heads, k_dim = k.shape[-2:]
    v_heads, d_v = v.shape[-2:]
    if k_dim != d_k:
        raise ValueError("q and k must have the same head size")
    if not isinstance(log_decay, torch.Tensor):
        raise TypeError("log_decay must be a CUDA tensor")
    if log_decay.dim() != 1:
        raise ValueError("log_decay must have shape [heads]")
    decay = _ptr_of("log_decay", log_decay, torch.float32, None, index)
    lens = _ptr_of("seq_lens", seq_lens, torch.int32, (batch,), index)
    if scale is None:
        scale = d_k ** -0.5 if d_k else 1.0
    block_len = seqlen if block_len is None else int(block_len)
    _int32("batch, seqlen and block_len", batch, seqlen, block_len)
    return LinattnArgs(batch, seqlen, block_len, log_decay.shape[0], q_heads,
                       k_heads, v_heads, d_k, d_v, 1 if reverse else 0, _DTYPE_CODE[dtype], scale,
                       q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, decay, lens)


def _dense(t: torch.Tensor, shape) -> torch.Tensor:
    """An uninitialised dense tensor of t's type and device."""
    return torch.empty_like(t) if t.shape == shape and t.is_contiguous() else t.new_empty(shape)


def _workspace(given: Optional[torch.Tensor], need: int, like: torch.Tensor, index: int):
    """(address or None, the tensor made here or None, bytes).  The tensor has to outlive the launch only: its memory is the
    working stream's."""
    if given is not None:
        return _ptr_of("workspace", given, given.dtype, None, index), None, given.numel() * given.element_size()
    if need == 0:
        return None, None, 0
    ws = like.new_empty(need, dtype=torch.uint8)
    return ws.data_ptr(), ws, need


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
    index = _first("q", q, 4)
    a = _linattn_args(q, k, v, log_decay, scale, block_len, reverse, seq_lens, tuple(q.shape[:2]), index)
    state = (a.batch, a.n_heads, a.d_k, a.d_v)
    shape = (a.batch, a.seqlen, a.n_heads, a.d_v)
    p0 = _ptr_of("h0", h0, torch.float32, state, index)
    p1 = _ptr_of("h_last", h_last, torch.float32, state, index)
    py = _ptr_of("y", y, q.dtype, shape, index)
    ref = ctypes.byref(a)
    place = _Place(stream, index)
    with place as raw:
        made_h = made_y = None
        if h_last is None and want_h_last:
            h_last = made_h = q.new_empty(state, dtype=torch.float32)
            p1 = h_last.data_ptr()
        if y is None:
            y = made_y = _dense(v, shape)
            py = y.data_ptr()
        ws, made, nbytes = _workspace(workspace, lib.r2l_linattn_workspace_size(ref), q, index)
        st = lib.r2l_linattn(ref, p0, p1, py, ws, nbytes, raw)
    place.give(made_h, made_y)
    if st != R2L_OK:
        _raise(st, "r2l_linattn")
    return y, h_last


def r2l_linattn_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, h: torch.Tensor, *,
                     scale: Optional[float] = None, h_out: Optional[torch.Tensor] = None,
                     y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of every sequence: q [b, q_heads, d_k], k [b, k_heads, d_k], v [b, v_heads, d_v], state h
    [b, heads, d_k, d_v] fp32, updated in place unless ``h_out`` is given.  Returns y [b, heads, d_v]."""
    lib = load_mixer()
    index = _first("q", q, 3)
    a = _linattn_args(q, k, v, log_decay, scale, None, False, None, (q.shape[0],), index)
    state = (a.batch, a.n_heads, a.d_k, a.d_v)
    shape = (a.batch, a.n_heads, a.d_v)
    if h is None:
        raise ValueError("h must be given")
    p0 = p1 = _ptr_of("h", h, torch.float32, state, index)
    if h_out is not None:
        p1 = _ptr_of("h_out", h_out, torch.float32, state, index)
    py = _ptr_of("y", y, q.dtype, shape, index)
    place = _Place(stream, index)
    with place as raw:
        made = None
        if y is None:
            y = made = _dense(v, shape)
            py = y.data_ptr()
        st = lib.r2l_linattn_step(ctypes.byref(a), p0, p1, py, raw)
    place.give(made)
    if st != R2L_OK:
        _raise(st, "r2l_linattn_step")
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
    index = _first("q", q, 4)
    a = _linattn_args(q, k, v, log_decay, scale, block_len, reverse, seq_lens, tuple(q.shape[:2]), index)
    state = (a.batch, a.n_heads, a.d_k, a.d_v)
    if dy is None:
        raise ValueError("dy must be given")
    pdy = _ptr_of("dy", dy, q.dtype, (a.batch, a.seqlen, a.n_heads, a.d_v), index)
    p0 = _ptr_of("h0", h0, torch.float32, state, index)
    pdh = _ptr_of("dh_last", dh_last, torch.float32, state, index)
    if want_dh0 is None:
        want_dh0 = h0 is not None
    ref = ctypes.byref(a)
    place = _Place(stream, index)
    with place as raw:
        dq, dk, dv = _dense(q, q.shape), _dense(k, k.shape), _dense(v, v.shape)
        dh0 = q.new_empty(state, dtype=torch.float32) if want_dh0 else None
        ws, made, nbytes = _workspace(workspace, lib.r2l_linattn_bwd_workspace_size(ref), q, index)
        st = lib.r2l_linattn_bwd(ref, pdy, p0, pdh, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(dh0), ws, nbytes, raw)
    place.give(dq, dk, dv, dh0)
    if st != R2L_OK:
        _raise(st, "r2l_linattn_bwd")
    return {"dq": dq, "dk": dk, "dv": dv, "dh0": dh0}


# ----------------------------------------------------------------------------- norm and rotation

def _rope_args(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved, index) -> QkNormRopeArgs:
    dtype = q.dtype
    tokens, q_heads, dim = q.shape
    qs, ks = _heads("q", q, dtype, (tokens,), index), _heads("k", k, dtype, (tokens,), index)
    if k.shape[2] != dim:
        raise ValueError("q and k must have the same head size")
    _int32("tokens", tokens, 0)
    wq = _ptr_of("q_weight", q_weight, torch.float32, (dim,), index)
    wk = _ptr_of("k_weight", k_weight, torch.float32, (dim,), index)
    rot, wide, pp, pf = 0, 0, None, None
    if inv_freq is not None:
        if isinstance(inv_freq, torch.Tensor) and inv_freq.dim() != 1:
            raise ValueError("inv_freq must have shape [rot_dim / 2]")
        pf = _ptr_of("inv_freq", inv_freq, torch.float32, None, index)
        rot = 2 * inv_freq.shape[0]
        if positions is None:
            raise ValueError("positions must be given with inv_freq")
        if not isinstance(positions, torch.Tensor):
            raise TypeError("positions must be a CUDA tensor")
        wide = 1 if positions.dtype is torch.int64 else 0
        if not wide and positions.dtype is not torch.int32:
            raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
        pp = _ptr_of("positions", positions, positions.dtype, (tokens,), index)
    return QkNormRopeArgs(tokens, q_heads, k.shape[1], dim, rot, 1 if interleaved else 0, wide, _DTYPE_CODE[dtype], eps,
                          q.data_ptr(), k.data_ptr(), qs, ks, wq, wk, pp, pf)


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
    index = _first("q", q, 3)
    a = _rope_args(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved, index)
    qs = 0 if q_out is None else _heads("q_out", q_out, q.dtype, (a.tokens,), index)
    ks = 0 if k_out is None else _heads("k_out", k_out, q.dtype, (a.tokens,), index)
    for name, o, t in (("q_out", q_out, q), ("k_out", k_out, k)):
        if o is not None and o.shape != t.shape:
            raise ValueError(f"{name} must have shape {tuple(t.shape)}, got {tuple(o.shape)}")
    made_q = made_k = None
    place = _Place(stream, index)
    with place as raw:
        if q_out is None:
            q_out = made_q = _dense(q, q.shape)
        if k_out is None:
            k_out = made_k = _dense(k, k.shape)
        st = lib.r2l_qk_norm_rope(ctypes.byref(a), q_out.data_ptr(), qs, k_out.data_ptr(), ks, raw)
    place.give(made_q, made_k)
    if st != R2L_OK:
        _raise(st, "r2l_qk_norm_rope")
    return q_out, k_out


def r2l_qk_norm_rope_bwd(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor],
                         k_weight: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                         inv_freq: Optional[torch.Tensor], dq_out: torch.Tensor, dk_out: torch.Tensor, *,
                         eps: float = 1e-6, interleaved: bool = False, workspace: Optional[torch.Tensor] = None,
                         stream=None) -> Dict[str, torch.Tensor]:
    """Gradients of r2l_qk_norm_rope (q and k: its inputs) given dq_out, dk_out: dq, dk in the inputs' type and
    dq_weight, dk_weight [d] fp32 (also where the weights were None, i.e. ones)."""
    lib = load_mixer()
    index = _first("q", q, 3)
    a = _rope_args(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved, index)
    if dq_out is None or dk_out is None:
        raise ValueError("dq_out and dk_out must be given")
    pdq = _ptr_of("dq_out", dq_out, q.dtype, q.shape, index)
    pdk = _ptr_of("dk_out", dk_out, q.dtype, k.shape, index)
    ref = ctypes.byref(a)
    place = _Place(stream, index)
    with place as raw:
        dq, dk = _dense(q, q.shape), _dense(k, k.shape)
        dqw, dkw = q.new_empty(a.head_dim, dtype=torch.float32), q.new_empty(a.head_dim, dtype=torch.float32)
        ws, made, nbytes = _workspace(workspace, lib.r2l_qk_norm_rope_bwd_workspace_size(ref), q, index)
        st = lib.r2l_qk_norm_rope_bwd(ref, pdq, pdk, dq.data_ptr(), dk.data_ptr(), dqw.data_ptr(), dkw.data_ptr(), ws, nbytes, raw)
    place.give(dq, dk, dqw, dkw)
    if st != R2L_OK:
        _raise(st, "r2l_qk_norm_rope_bwd")
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def r2l_mixer_device_status(stream=None) -> int:
    """Synchronise and read/clear this library's device status word (R2L_OK or R2L_ERR_TIMEOUT)."""
    with _Place(stream, torch.cuda.current_device()) as raw:
        return int(load_mixer().r2l_mixer_device_status(raw))


def r2l_mixer_abi_version() -> int:
    return int(load_mixer().r2l_mixer_abi_version())
