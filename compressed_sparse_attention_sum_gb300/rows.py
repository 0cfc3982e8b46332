"""Python binding of the row calls (include/csa_rows.h): layer and RMS norms and
rotary positions of the rows that a layer works on, and their gradients.

Argument marshalling only, as in csa.py: each function checks the tensors it is
given, allocates missing outputs and workspaces with PyTorch and calls the
entry point of the same name in libcsa.so on the current stream of the tensors'
device.  There is no fallback: a missing library or a failed call raises.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import csa
from .csa import CSAError  # noqa: F401  (re-exported)
from .serve import _DT, _F32, _I32, _elsewhere, _empty, _on, _optional, _refuse, _workspace

_c_int, _c_ll, _c_p, _c_f, _c_sz, _c_d = (ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p,
                                          ctypes.c_float, ctypes.c_size_t, ctypes.c_double)

CSA_NORM_RMS, CSA_NORM_LAYER = 1, 2
CSA_ROPE_INTERLEAVED, CSA_ROPE_HALF = 0, 1
_LAYOUTS = {"interleaved": CSA_ROPE_INTERLEAVED, "half": CSA_ROPE_HALF}
_SCALINGS = {"plain": 0, "linear": 1, "by_parts": 2}


class _RopeStruct(ctypes.Structure):
    _fields_ = [("turns", _c_p), ("dim", _c_int), ("first", _c_int), ("layout", _c_int),
                ("scale", _c_f)]


class _Strides(ctypes.Structure):
    _fields_ = [("batch", _c_ll), ("token", _c_ll), ("head", _c_ll)]


SIGNATURES = {
    "csa_norm": (_c_int, [_c_p, _c_ll, _c_int, _c_int, _c_p, _c_p, _c_f, _c_p, _c_ll, _c_ll,
                          _c_int, _c_p]),
    "csa_norm_bwd_workspace_size": (_c_sz, [_c_ll, _c_int, _c_int, _c_int]),
    "csa_norm_bwd": (_c_int, [_c_p, _c_ll, _c_int, _c_int, _c_p, _c_f, _c_p, _c_ll, _c_int, _c_p,
                              _c_ll, _c_int, _c_p, _c_p, _c_ll, _c_int, _c_p, _c_sz, _c_p]),
    "csa_rope_freqs": (_c_int, [_c_int, _c_d, _c_int, _c_d, _c_d, _c_d, _c_d, _c_p]),
    "csa_rope_turns": (_c_int, [_c_p, _c_int, _c_p]),
    "csa_rope": (_c_int, [_c_p, _c_p, _c_int, _c_p, _c_ll, _c_p, _c_int, _c_p, _c_p]
                 + [_c_int] * 4 + [_c_p]),
    "csa_rope_bwd": (_c_int, [_c_p, _c_p, _c_int, _c_p, _c_ll, _c_p, _c_int, _c_p, _c_p]
                     + [_c_int] * 5 + [_c_p]),
    "csa_norm_rope": (_c_int, [_c_p, _c_p, _c_int, _c_int, _c_p, _c_p, _c_f, _c_p, _c_ll, _c_p,
                               _c_p, _c_p] + [_c_int] * 4 + [_c_p]),
    "csa_norm_rope_bwd": (_c_int, [_c_p, _c_p, _c_int, _c_int, _c_p, _c_f, _c_p, _c_ll, _c_p,
                                   _c_p, _c_p, _c_int, _c_p, _c_p, _c_int, _c_p, _c_p]
                          + [_c_int] * 4 + [_c_p, _c_sz, _c_p]),
    "csa_compress_decode": (_c_int, [_c_p, _c_ll, _c_ll, _c_p, _c_ll, _c_ll, _c_int, _c_p, _c_p,
                                     _c_int, _c_p, _c_int, _c_p, _c_p, _c_f, _c_p, _c_p, _c_ll,
                                     _c_p, _c_p] + [_c_int] * 6 + [_c_p]),
}

_declared = None


def load_library():
    """libcsa.so with the row calls' C signatures declared."""
    global _declared
    lib = csa.load_library()
    if _declared is not lib:
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _declared = lib
    return lib


_entries = {}


def _entry(name):
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(load_library(), name)
    return fn


def _call(name, dev, stream, *args):
    """Call an entry point with device dev current, on `stream` or on dev's current stream."""
    fn = _entries.get(name) or _entry(name)
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _call(name, dev, stream, *args)
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, expected cuda:{dev}")
    else:
        s = stream.cuda_stream
    code = fn(*args, s)
    if code != 0:
        raise CSAError(name, code)


_INT_MAX = 2 ** 31 - 1     # ctypes would pass a larger int's low 32 bits


def _fits(name, largest):
    if largest > _INT_MAX:
        raise ValueError(f"{name} has a size of 2^31 or more")


def _kind(kind):
    """A norm's kind as the entry points take it (0: none), which refuse the other small ones."""
    if kind >> 2:
        raise ValueError("kind must be CSA_NORM_RMS or CSA_NORM_LAYER")
    return kind


class CsaRope:
    """A rotation: `turns` (csa_rope_turns, one of each channel pair) on the device, the
    first turned channel, the pairs' layout ("interleaved" or "half") and a factor on
    the turned channels.  Made once and given to every call; immutable."""

    __slots__ = ("turns", "first", "layout", "scale", "dim", "_struct", "_pointer", "_device")

    def __init__(self, turns: torch.Tensor, first: int = 0, layout: str = "interleaved",
                 scale: float = 1.0):
        if not turns.is_cuda:
            raise ValueError("turns must be a CUDA tensor")
        if turns.dtype != torch.int64 or turns.ndim != 1 or not turns.is_contiguous():
            raise TypeError("turns must be a contiguous int64 vector (csa_rope_turns)")
        if layout not in _LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}")
        if not 0 <= int(first) <= _INT_MAX:
            raise ValueError("first must be a channel of the row")
        _fits("turns", 2 * turns.shape[0])
        put = super().__setattr__
        put("turns", turns)
        put("first", int(first))
        put("layout", layout)
        put("scale", float(scale))
        put("dim", 2 * turns.shape[0])
        put("_struct", _RopeStruct(turns.data_ptr(), self.dim, self.first, _LAYOUTS[layout],
                                   self.scale))
        put("_pointer", ctypes.addressof(self._struct))
        put("_device", turns.get_device())

    def __setattr__(self, name, value):
        raise AttributeError("a CsaRope does not change")


def csa_rope_freqs(dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                   original_len: float = 0.0, beta_fast: float = 32.0,
                   beta_slow: float = 1.0) -> torch.Tensor:
    """The dim / 2 frequencies of a rotation (radians a position), fp64 on the host:
    "plain", "linear" (divided by factor) or "by_parts" (low ones divided, high ones
    kept; contexts of original_len positions stretched by factor)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    _fits("dim", abs(int(dim)))
    out = torch.empty(max(0, int(dim) // 2), dtype=torch.float64)
    code = load_library().csa_rope_freqs(int(dim), float(base), _SCALINGS[scaling], float(factor),
                                         float(original_len), float(beta_fast), float(beta_slow),
                                         out.data_ptr() or None)
    if code != 0:
        raise CSAError("csa_rope_freqs", code)
    return out


def csa_rope_turns(freqs, device="cuda") -> torch.Tensor:
    """Frequencies (radians a position) as int64 parts of a turn on `device`."""
    freqs = torch.as_tensor(freqs, dtype=torch.float64, device="cpu")
    if freqs.ndim != 1:
        raise ValueError("freqs must be a vector")
    _fits("freqs", freqs.shape[0])
    freqs = freqs.contiguous()
    out = torch.empty(freqs.shape[0], dtype=torch.int64)
    code = load_library().csa_rope_turns(freqs.data_ptr() or None, freqs.shape[0],
                                         out.data_ptr() or None)
    if code != 0:
        raise CSAError("csa_rope_turns", code)
    return out.to(device)


def _new(shape, dtype, dev):
    """An uninitialised contiguous tensor on device dev."""
    strides, n = [], 1
    for size in reversed(shape):
        strides.append(n)
        n *= size
    return _empty(tuple(shape), tuple(reversed(strides)), dtype, dev)


def _zeros(shape, strides, dtype, dev):
    return torch.zeros(shape, dtype=dtype, device=f"cuda:{dev}")


def _first(t, name):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"unsupported dtype {t.dtype} of {name} (bf16 or fp32)")
    return dev, dt


def _like(t, name, shape, dev):
    """dtype code of another tensor of a call's rows."""
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"unsupported dtype {t.dtype} of {name} (bf16 or fp32)")
    if t.get_device() != dev or t.shape != shape:
        _refuse(dev, **{name: (t, t.dtype, shape)})
    return dt


def _row_stride(t, name, n):
    """Row stride of [..., n] rows that one stride reaches."""
    if t.is_contiguous():
        return n
    strides, shape = t.stride(), t.shape
    if len(strides) == 2 and strides[1] == 1:
        return strides[0]
    if t.numel() == 0:
        return n
    if strides[-1] != 1:
        raise ValueError(f"{name} rows must be contiguous")
    step, last = None, None           # the stride of the rows; what the next dimension out has
    for size, st in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if size == 1:
            continue
        if step is None:
            step = st
        elif st != last:
            raise ValueError(f"{name} rows must lie one row stride apart")
        last = st * size
    return n if step is None else step


_strides_of = {}


def _strides(t, name):
    """The strides of rows [b, s, H, d] (or [b, s, d]), by reference; the reference keeps
    them alive."""
    key = t.stride()
    if len(key) == 3:
        key = (*key[:2], 0, key[2])
    got = _strides_of.get(key)
    if got is None:
        got = ctypes.byref(_Strides(*key[:3]))
        if key[3] != 1:
            if t.numel():
                raise ValueError(f"{name} rows must be contiguous")
            return got
        if len(_strides_of) >= 4096:
            _strides_of.clear()
        _strides_of[key] = got
    return got


def _vector(t, name, n, dev):
    if t is None:
        return None
    if not (t.get_device() == dev and t.dtype is _F32 and t.shape == (n,) and t.is_contiguous()):
        _refuse(dev, **{name: (t, _F32, (n,))})
    return t.data_ptr()


def _positions(pos, b, s, dev):
    """Pointer and batch stride of positions [b, s] or [s]."""
    if pos is None:
        return None, 0
    shape, strides = pos.shape, pos.stride()
    if (pos.get_device() != dev or pos.dtype is not _I32
            or (shape != (b, s) and shape != (s,))):
        _refuse(dev, pos=(pos, _I32, (s,) if len(shape) == 1 else (b, s)))
    if s > 1 and strides[-1] != 1:
        raise ValueError("pos must be contiguous along the tokens")
    return pos.data_ptr(), (strides[0] if len(shape) == 2 and b > 1 else 0)


def _heads(shape, name):
    """b, s, H, d of [b, s, H, d] or [b, s, d]."""
    if len(shape) == 4:
        _fits(name, max(shape))
        return shape
    if len(shape) == 3:
        _fits(name, max(shape))
        b, s, d = shape
        return b, s, 1, d
    raise ValueError(f"{name} must be [b, s, H, d] or [b, s, d]")


def _rope(rope, dev):
    if not isinstance(rope, CsaRope):
        raise TypeError("rope must be a CsaRope")
    if rope._device != dev:
        raise ValueError(f"the rotation is on cuda:{rope._device}, expected cuda:{dev}")
    return rope._pointer


def csa_norm(x: torch.Tensor, kind: int, weight: Optional[torch.Tensor] = None,
             bias: Optional[torch.Tensor] = None, eps: float = 1e-6,
             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Norm (CSA_NORM_RMS or CSA_NORM_LAYER) of the rows of x [..., n] (bf16 or fp32; rows
    contiguous, one row stride), times weight [n] fp32, plus bias [n] fp32.  out may be x.
    """
    if stream is not None and _elsewhere(stream, x):
        return _on(stream, csa_norm, x, kind, weight, bias, eps, out)
    dev, dt = _first(x, "x")
    shape = x.shape
    if not shape:
        raise ValueError("x must be [..., n]")
    n = shape[-1]
    _fits("x", n)
    if out is None:
        out = _new(shape, x.dtype, dev)
    elif out.dtype is not x.dtype or out.shape != shape or out.get_device() != dev:
        _refuse(dev, out=(out, x.dtype, shape))
    _call("csa_norm", dev, stream, x.data_ptr(), _row_stride(x, "x", n), dt, _kind(kind),
          _vector(weight, "weight", n, dev), _vector(bias, "bias", n, dev), float(eps),
          out.data_ptr(), _row_stride(out, "out", n), x.numel() // n if n else 0, n)
    return out


def csa_norm_bwd_workspace_size(rows: int, n: int, want_dweight: bool = True,
                                want_dbias: bool = False) -> int:
    """Workspace bytes of csa_norm_bwd, and of csa_norm_rope_bwd with b * s * H rows."""
    _fits("a row", n)
    return _entry("csa_norm_bwd_workspace_size")(rows, n, 1 if want_dweight else 0,
                                                 1 if want_dbias else 0)


def _bwd_workspace(workspace, rows, n, dweight, dbias, dev):
    """The tensor, pointer and size of a backward call's workspace."""
    if workspace is not None:
        return _workspace(workspace, 0, dev)
    if dweight is None and dbias is None:
        return None, None, 0
    nbytes = csa_norm_bwd_workspace_size(rows, n, dweight is not None, dbias is not None)
    if nbytes == 0:
        return None, None, 0
    ws = _empty((nbytes,), (1,), torch.uint8, dev)
    return ws, ws.data_ptr(), nbytes


def _sums(weight, has_bias, dweight, dbias, n, dev):
    """dweight and dbias of a backward call (None: not wanted)."""
    if dweight is not None:
        _optional(dweight, "dweight", _F32, (n,), dev)
    elif weight is not None:
        dweight = _empty((n,), (1,), _F32, dev)
    if dbias is not None:
        _optional(dbias, "dbias", _F32, (n,), dev)
    elif has_bias:
        dbias = _empty((n,), (1,), _F32, dev)
    return dweight, dbias


def csa_norm_bwd(x: torch.Tensor, dout: torch.Tensor, kind: int,
                 weight: Optional[torch.Tensor] = None, eps: float = 1e-6, has_bias: bool = False,
                 dx: Optional[torch.Tensor] = None, dweight: Optional[torch.Tensor] = None,
                 dbias: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None
                 ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradient of csa_norm: (dx, dweight, dbias).

    dout and dx are [..., n] like x, each bf16 or fp32 (dx: x's dtype where it is not
    given; it may be dout or x).  dweight [n] fp32 is returned where the norm has a
    weight, dbias [n] fp32 where has_bias, and either where a tensor for it is given.
    """
    if stream is not None and _elsewhere(stream, x):
        return _on(stream, csa_norm_bwd, x, dout, kind, weight, eps, has_bias, dx, dweight, dbias,
                   workspace)
    dev, dt = _first(x, "x")
    shape = x.shape
    if not shape:
        raise ValueError("x must be [..., n]")
    n = shape[-1]
    _fits("x", n)
    rows = x.numel() // n if n else 0
    g_dt = _like(dout, "dout", shape, dev)
    if dx is None:
        dx = _new(shape, x.dtype, dev)
    dx_dt = _like(dx, "dx", shape, dev)
    w = _vector(weight, "weight", n, dev)
    dweight, dbias = _sums(weight, has_bias, dweight, dbias, n, dev)
    keep, ws, nbytes = _bwd_workspace(workspace, rows, n, dweight, dbias, dev)
    _call("csa_norm_bwd", dev, stream, x.data_ptr(), _row_stride(x, "x", n), dt, _kind(kind), w,
          float(eps), dout.data_ptr(), _row_stride(dout, "dout", n), g_dt, dx.data_ptr(),
          _row_stride(dx, "dx", n), dx_dt, None if dweight is None else dweight.data_ptr(),
          None if dbias is None else dbias.data_ptr(), rows, n, ws, nbytes)
    return dx, dweight, dbias


def csa_rope(x: torch.Tensor, rope: CsaRope, pos: Optional[torch.Tensor] = None,
             inverse: bool = False, out: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """Rows x [b, s, H, d] or [b, s, d] (bf16 or fp32; channels contiguous, any strides of
    16-byte multiples) turned by their token's position: pos [b, s] or [s] int32, or the
    token's index.  inverse: turned back.  out may be x (the turned channels alone are
    then read and written)."""
    if stream is not None and _elsewhere(stream, x):
        return _on(stream, csa_rope, x, rope, pos, inverse, out)
    dev, dt = _first(x, "x")
    shape = x.shape
    b, s, H, d = _heads(shape, "x")
    if out is None:
        out = _new(shape, x.dtype, dev)
    elif out.dtype is not x.dtype or out.shape != shape or out.get_device() != dev:
        _refuse(dev, out=(out, x.dtype, shape))
    p, ps = _positions(pos, b, s, dev)
    _call("csa_rope", dev, stream, x.data_ptr(), _strides(x, "x"), dt, p, ps,
          _rope(rope, dev), 1 if inverse else 0, out.data_ptr(), _strides(out, "out"), b, s,
          H, d)
    return out


def csa_rope_bwd(dout: torch.Tensor, rope: CsaRope, pos: Optional[torch.Tensor] = None,
                 inverse: bool = False, dx: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Gradient of csa_rope (rope, pos and inverse as it had them): dout [b, s, H, d] or
    [b, s, d], bf16 or fp32; dx, of dout's dtype where it is not given, may be dout."""
    if stream is not None and _elsewhere(stream, dout):
        return _on(stream, csa_rope_bwd, dout, rope, pos, inverse, dx)
    dev, dt = _first(dout, "dout")
    shape = dout.shape
    b, s, H, d = _heads(shape, "dout")
    if dx is None:
        dx = _new(shape, dout.dtype, dev)
    dx_dt = _like(dx, "dx", shape, dev)
    p, ps = _positions(pos, b, s, dev)
    _call("csa_rope_bwd", dev, stream, dout.data_ptr(), _strides(dout, "dout"), dt, p, ps,
          _rope(rope, dev), 1 if inverse else 0, dx.data_ptr(), _strides(dx, "dx"), dx_dt, b,
          s, H, d)
    return dx


def csa_norm_rope(x: torch.Tensor, kind: int, rope: CsaRope, pos: Optional[torch.Tensor] = None,
                  weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  eps: float = 1e-6, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """csa_norm of each row's d channels (weight and bias [d] fp32), then csa_rope, rounded
    once; x [b, s, H, d] or [b, s, d].  out may be x."""
    if stream is not None and _elsewhere(stream, x):
        return _on(stream, csa_norm_rope, x, kind, rope, pos, weight, bias, eps, out)
    dev, dt = _first(x, "x")
    shape = x.shape
    b, s, H, d = _heads(shape, "x")
    if out is None:
        out = _new(shape, x.dtype, dev)
    elif out.dtype is not x.dtype or out.shape != shape or out.get_device() != dev:
        _refuse(dev, out=(out, x.dtype, shape))
    p, ps = _positions(pos, b, s, dev)
    _call("csa_norm_rope", dev, stream, x.data_ptr(), _strides(x, "x"), dt, _kind(kind),
          _vector(weight, "weight", d, dev), _vector(bias, "bias", d, dev), float(eps), p, ps,
          _rope(rope, dev), out.data_ptr(), _strides(out, "out"), b, s, H, d)
    return out


def csa_norm_rope_bwd(x: torch.Tensor, dout: torch.Tensor, kind: int, rope: CsaRope,
                      pos: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                      eps: float = 1e-6, has_bias: bool = False,
                      dx: Optional[torch.Tensor] = None, dweight: Optional[torch.Tensor] = None,
                      dbias: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None
                      ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradient of csa_norm_rope: (dx, dweight, dbias), as csa_norm_bwd gives them; dweight
    and dbias [d] are summed over all rows and heads."""
    if stream is not None and _elsewhere(stream, x):
        return _on(stream, csa_norm_rope_bwd, x, dout, kind, rope, pos, weight, eps, has_bias, dx,
                   dweight, dbias, workspace)
    dev, dt = _first(x, "x")
    shape = x.shape
    b, s, H, d = _heads(shape, "x")
    g_dt = _like(dout, "dout", shape, dev)
    if dx is None:
        dx = _new(shape, x.dtype, dev)
    dx_dt = _like(dx, "dx", shape, dev)
    w = _vector(weight, "weight", d, dev)
    dweight, dbias = _sums(weight, has_bias, dweight, dbias, d, dev)
    keep, ws, nbytes = _bwd_workspace(workspace, b * s * H, d, dweight, dbias, dev)
    p, ps = _positions(pos, b, s, dev)
    _call("csa_norm_rope_bwd", dev, stream, x.data_ptr(), _strides(x, "x"), dt, _kind(kind), w,
          float(eps), p, ps, _rope(rope, dev), dout.data_ptr(), _strides(dout, "dout"), g_dt,
          dx.data_ptr(), _strides(dx, "dx"), dx_dt,
          None if dweight is None else dweight.data_ptr(),
          None if dbias is None else dbias.data_ptr(), b, s, H, d, ws, nbytes)
    return dx, dweight, dbias


def csa_compress_decode(kv: torch.Tensor, score: torch.Tensor, kv_ring: torch.Tensor,
                        score_ring: torch.Tensor, seq_lens: torch.Tensor, ratio: int,
                        coff: int = 1, kind: int = 0, weight: Optional[torch.Tensor] = None,
                        bias: Optional[torch.Tensor] = None, eps: float = 1e-6,
                        rope: Optional[CsaRope] = None,
                        out: Optional[torch.Tensor] = None, first: Optional[torch.Tensor] = None,
                        counts: Optional[torch.Tensor] = None, stream=None
                        ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The compressor for the newest s_q tokens of each sequence.

    kv [b, s_q, d] and score [b, s_q, d or 1] (bf16 or fp32, rows contiguous) are the new
    tokens' rows, seq_lens [b] int32 counts all tokens; kv_ring [b, R, d] and score_ring
    [b, R, d or 1] keep the newest rows (R >= coff * ratio - 1 + s_q for calls whose tokens
    may be taken back, R >= coff * ratio at least) and take the new ones.  The blocks that
    the tokens complete are pooled (coff blocks a window), normalised (kind CSA_NORM_RMS or
    CSA_NORM_LAYER, 0: not) and turned (rope).  Returns
    (out [b, ceil(s_q / ratio), d], first [b], counts [b]): x, pos0 and counts of
    csa_cache_write; rows of out from counts on are left as they were.  Without new tokens
    (s_q 0) nothing is written; first and counts are zeros unless they were given.
    """
    if stream is not None and _elsewhere(stream, kv):
        return _on(stream, csa_compress_decode, kv, score, kv_ring, score_ring, seq_lens, ratio,
                   coff, kind, weight, bias, eps, rope, out, first, counts)
    dev, dt = _first(kv, "kv")
    if kv.ndim != 3:
        raise ValueError("kv must be [b, s_q, d]")
    b, s_q, d = kv.shape
    if score.ndim != 3 or kv_ring.ndim != 3 or ratio < 1:
        raise ValueError("score and kv_ring must have three dimensions, ratio be at least 1")
    dtype, sw, R = kv.dtype, score.shape[2], kv_ring.shape[1]
    _fits("kv, a ring or a block", max(b, s_q, d, sw, R, ratio, coff))
    if not (score.dtype is dtype and kv_ring.dtype is dtype and score_ring.dtype is dtype
            and seq_lens.dtype is _I32 and score.get_device() == dev
            and kv_ring.get_device() == dev and score_ring.get_device() == dev
            and seq_lens.get_device() == dev and score.shape == (b, s_q, sw)
            and kv_ring.shape == (b, R, d) and score_ring.shape == (b, R, sw)
            and seq_lens.shape == (b,) and kv_ring.is_contiguous() and score_ring.is_contiguous()
            and seq_lens.is_contiguous()):
        if score.dtype is not dtype or score.shape != (b, s_q, sw) or score.get_device() != dev:
            _refuse(dev, score=(score, dtype, (b, s_q, sw)))
        _refuse(dev, kv_ring=(kv_ring, dtype, (b, R, d)), score_ring=(score_ring, dtype, (b, R, sw)),
                seq_lens=(seq_lens, _I32, (b,)))
    kb, kr, kc = kv.stride()
    sb, sr, sc = score.stride()
    if ((kc != 1 and d > 1) or (sc != 1 and sw > 1)) and b and s_q:
        raise ValueError("rows of kv and score must be contiguous")
    w, bp = _vector(weight, "weight", d, dev), _vector(bias, "bias", d, dev)
    turned = None if rope is None else _rope(rope, dev)
    blocks = -(-s_q // ratio)
    if out is None:
        out, ob = _empty((b, blocks, d), (blocks * d, d, 1), dtype, dev), blocks * d
    else:
        if not (out.dtype is dtype and out.shape == (b, blocks, d) and out.get_device() == dev):
            _refuse(dev, out=(out, dtype, (b, blocks, d)))
        ob, orow, oc = out.stride()
        if blocks and b and (oc != 1 or (blocks > 1 and orow != d)):
            raise ValueError("out rows must be packed")
    made = _empty if s_q else _zeros
    if first is None:
        first = made((b,), (1,), _I32, dev)
    else:
        _optional(first, "first", _I32, (b,), dev)
    if counts is None:
        counts = made((b,), (1,), _I32, dev)
    else:
        _optional(counts, "counts", _I32, (b,), dev)
    _call("csa_compress_decode", dev, stream, kv.data_ptr(), kb, kr, score.data_ptr(),
          sb, sr, sw, kv_ring.data_ptr(), score_ring.data_ptr(), R, seq_lens.data_ptr(), _kind(kind), w,
          bp, float(eps), turned, out.data_ptr(), ob, first.data_ptr(),
          counts.data_ptr(), b, s_q, d, ratio, coff, dt)
    return out, first, counts
