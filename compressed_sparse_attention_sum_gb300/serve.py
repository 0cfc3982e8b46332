"""Python binding of the serving calls (include/csa_serve.h): the quantised
paged cache, and the indexer and attention of single tokens over it.

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
from .csa import CSA_BF16, CSA_FP32, CSAError  # noqa: F401  (CSAError: re-exported)

_c_int, _c_ll, _c_p, _c_f, _c_sz = (ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p,
                                    ctypes.c_float, ctypes.c_size_t)
_DT = {torch.bfloat16: CSA_BF16, torch.float32: CSA_FP32}
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8

SIGNATURES = {
    "csa_cache_page_bytes": (_c_sz, [_c_int] * 3),
    "csa_cache_write": (_c_int, [_c_p, _c_ll, _c_ll, _c_int, _c_p, _c_p, _c_p, _c_p]
                        + [_c_int] * 7 + [_c_p]),
    "csa_cache_read": (_c_int, [_c_p] * 5 + [_c_ll, _c_ll, _c_int] + [_c_int] * 7 + [_c_p]),
    "csa_indexer_topk_decode_workspace_size": (_c_sz, [_c_int] * 5),
    "csa_indexer_topk_decode": (_c_int, [_c_p] * 6 + [_c_int] * 10 + [_c_int, _c_p, _c_sz, _c_p]),
    "csa_attn_decode_workspace_size": (_c_sz, [_c_int] * 6),
    "csa_attn_decode": (_c_int, [_c_p] * 7 + [_c_f, _c_p, _c_p] + [_c_int] * 12
                        + [_c_int, _c_p, _c_sz, _c_p]),
}

_declared = None
_page_bytes = {}


def load_library():
    """libcsa.so with the serving calls' C signatures declared."""
    global _declared
    lib = csa.load_library()
    if _declared is not lib:
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _declared = lib
    return lib


# A decode step makes these calls for every layer and token, with kernels of a
# few microseconds, so the checks cost as little as they can where nothing is
# wrong: one condition over all of a call's tensors, and _refuse names the first
# that is at fault when it fails.

def _refuse(dev, **tensors):
    """Raise for the first (tensor, dtype, shape) that is not a contiguous CUDA
    tensor of that dtype and shape on device dev."""
    for name, (t, dtype, shape) in tensors.items():
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    raise ValueError("arguments do not agree")


# torch's allocation without its dispatcher, as its compiler's generated code
# calls it: 2 us of a call instead of 4 (torch.empty) or 7 (new_empty).  Only
# where no dispatch mode is active, so that one sees every output's allocation.
_modes = getattr(torch._C, "_len_torch_dispatch_stack", None)
_empty_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None),
                         "_empty_strided_cuda", None) if _modes is not None else None


def _empty(shape, stride, dtype, dev):
    """An uninitialised contiguous tensor on device dev."""
    if _empty_strided is not None and _modes() == 0 and torch._C._cuda_getDevice() == dev:
        return _empty_strided(shape, stride, dtype)
    return torch.empty(shape, dtype=dtype, device=f"cuda:{dev}")


def _optional(t, name, dtype, shape, dev):
    if not (t.get_device() == dev and t.dtype is dtype and t.shape == shape
            and t.is_contiguous()):
        _refuse(dev, **{name: (t, dtype, shape)})


def _first(t, name, dims):
    """The device index and dtype code of a call's main tensor."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")
    if t.ndim != len(dims):
        raise ValueError(f"{name} must be [{', '.join(dims)}]")
    return dev, dt


def _columns(t, name):
    """Columns of a two-dimensional tensor, at least one."""
    if t.ndim != 2 or t.shape[1] < 1:
        raise ValueError(f"{name} must have two dimensions and at least one column")
    return t.shape[1]


def _workspace(ws, nbytes, dev):
    """Pointer and size of the workspace; the tensor is returned to be kept alive."""
    if ws is None:
        if nbytes == 0:
            return None, None, 0
        ws = torch.empty(nbytes, dtype=_U8, device=f"cuda:{dev}")
    elif not (ws.get_device() == dev and ws.is_contiguous()):
        _refuse(dev, workspace=(ws, ws.dtype, ws.shape))
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _elsewhere(stream, t):
    """Whether `stream` is another stream of t's device than the current one."""
    if stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, expected {t.device}")
    return stream != torch.cuda.current_stream(t.device)


def _on(stream, call, *args):
    """The call with `stream` current: what it allocates belongs to that stream too,
    and is not handed to another while its kernels run."""
    with torch.cuda.stream(stream):
        return call(*args, stream=stream)


def _call(name, dev, stream, *args):
    """Call an entry point with device dev current, on `stream` or on dev's current stream."""
    fn = getattr(_declared or load_library(), name)
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


def csa_cache_page_bytes(page_size: int, d: int, bits: int) -> int:
    """Bytes of one page of `page_size` rows of d channels in 4 or 8 bits."""
    key = (page_size, d, bits)
    n = _page_bytes.get(key)
    if n is None:
        n = int(load_library().csa_cache_page_bytes(int(page_size), int(d), int(bits)))
        if n == 0:
            raise ValueError(f"no cache format with pages of {page_size} rows, {d} channels and "
                             f"{bits} bits (page_size % 16 == 0, d % 32 == 0, d <= 512, bits 4 "
                             "or 8)")
        _page_bytes[key] = n
    return n


def _rows_args(x, name, cache, table, pos0, page_size, bits, counts):
    dev, dt = _first(x, name, ("b", "s", "d"))
    b, s, d = x.shape
    bs, rs, cs = x.stride()
    if cs != 1 and b and s:
        raise ValueError(f"{name} rows must be contiguous")
    want = csa_cache_page_bytes(page_size, d, bits)
    n_pages, row = cache.shape if cache.ndim == 2 else (0, -1)
    P = _columns(table, "table")
    if not (row == want and cache.dtype is _U8 and table.dtype is _I32 and pos0.dtype is _I32
            and cache.get_device() == dev and table.get_device() == dev
            and pos0.get_device() == dev and table.shape[0] == b and pos0.shape == (b,)
            and cache.is_contiguous() and table.is_contiguous() and pos0.is_contiguous()):
        _refuse(dev, cache=(cache, _U8, (n_pages, want)), table=(table, _I32, (b, P)),
                pos0=(pos0, _I32, (b,)))
    if counts is not None:
        _optional(counts, "counts", _I32, (b,), dev)
    return dev, dt, b, s, d, bs, rs, P, n_pages


def csa_cache_write(x: torch.Tensor, cache: torch.Tensor, table: torch.Tensor, pos0: torch.Tensor,
                    page_size: int, bits: int, counts: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """Quantise rows into the cache: row i < counts[s] (None: all) of
    x [b, s, d] (bf16 or fp32, rows contiguous, any row and batch stride of
    16-byte multiples) goes to position pos0[s] + i of sequence s.

    cache [n_pages, csa_cache_page_bytes(page_size, d, bits)] uint8, table
    [b, P] int32 page ids, pos0 and counts [b] int32.  Positions run through
    the P * page_size slots as through a ring.  Returns cache.
    """
    dev, dt, b, s, d, bs, rs, P, n_pages = _rows_args(x, "x", cache, table, pos0, page_size, bits,
                                                      counts)
    _call("csa_cache_write", dev, stream, x.data_ptr(), bs, rs, dt, table.data_ptr(),
          pos0.data_ptr(), None if counts is None else counts.data_ptr(), cache.data_ptr(), b, s,
          d, P, n_pages, page_size, bits)
    return cache


def csa_cache_read(cache: torch.Tensor, table: torch.Tensor, pos0: torch.Tensor,
                   out: torch.Tensor, page_size: int, bits: int,
                   counts: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Read the rows at positions pos0[s] .. pos0[s] + counts[s] - 1 into
    out [b, s, d] (bf16 or fp32, rows contiguous), exactly as the codes stand
    for them; rows past counts[s] are left as they were.  Returns out."""
    dev, dt, b, s, d, bs, rs, P, n_pages = _rows_args(out, "out", cache, table, pos0, page_size,
                                                      bits, counts)
    _call("csa_cache_read", dev, stream, cache.data_ptr(), table.data_ptr(), pos0.data_ptr(),
          None if counts is None else counts.data_ptr(), out.data_ptr(), bs, rs, dt, b, s, d, P,
          n_pages, page_size, bits)
    return out


def csa_indexer_topk_decode_workspace_size(b: int, s_q: int, H_I: int, d_I: int,
                                           slots: int) -> int:
    """Workspace bytes; slots = P * page_size of the page table."""
    return int(load_library().csa_indexer_topk_decode_workspace_size(b, s_q, H_I, d_I, slots))


def csa_indexer_topk_decode(q_I: torch.Tensor, cache: torch.Tensor, table: torch.Tensor,
                            w: torch.Tensor, seq_lens: torch.Tensor, topk: int, ratio: int,
                            page_size: int, bits: int,
                            workspace: Optional[torch.Tensor] = None,
                            out_idx: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Exact top-k blocks of the newest s_q tokens of each sequence.

    q_I [b, s_q, H_I, d_I], w [b, s_q, H_I] fp32, seq_lens [b] int32 (tokens
    of each sequence, the s_q newest included), table [b, P] the index keys'
    pages (block j at position j).  Returns idx [b, s_q, topk] int32:
    ascending, -1 behind the min(topk, vis) blocks.
    """
    if stream is not None and _elsewhere(stream, q_I):
        return _on(stream, csa_indexer_topk_decode, q_I, cache, table, w, seq_lens, topk, ratio,
                   page_size, bits, workspace, out_idx)
    dev, dt = _first(q_I, "q_I", ("b", "s_q", "H_I", "d_I"))
    b, s_q, H, d = q_I.shape
    want = csa_cache_page_bytes(page_size, d, bits)
    n_pages, row = cache.shape if cache.ndim == 2 else (0, -1)
    P = _columns(table, "table")
    if not (row == want and cache.dtype is _U8 and table.dtype is _I32 and w.dtype is _F32
            and seq_lens.dtype is _I32 and cache.get_device() == dev and table.get_device() == dev
            and w.get_device() == dev and seq_lens.get_device() == dev and table.shape[0] == b
            and w.shape == (b, s_q, H) and seq_lens.shape == (b,) and q_I.is_contiguous()
            and cache.is_contiguous() and table.is_contiguous() and w.is_contiguous()
            and seq_lens.is_contiguous()):
        _refuse(dev, q_I=(q_I, q_I.dtype, q_I.shape), cache=(cache, _U8, (n_pages, want)),
                table=(table, _I32, (b, P)), w=(w, _F32, (b, s_q, H)),
                seq_lens=(seq_lens, _I32, (b,)))
    if topk < 1:
        raise ValueError("topk must be at least 1")
    if out_idx is None:
        out_idx = _empty((b, s_q, topk), (s_q * topk, topk, 1), _I32, dev)
    else:
        _optional(out_idx, "out_idx", _I32, (b, s_q, topk), dev)
    nbytes = (csa_indexer_topk_decode_workspace_size(b, s_q, H, d, P * page_size)
              if workspace is None else 0)
    keep, ws, nbytes = _workspace(workspace, nbytes, dev)
    _call("csa_indexer_topk_decode", dev, stream, q_I.data_ptr(), cache.data_ptr(),
          table.data_ptr(), w.data_ptr(), seq_lens.data_ptr(), out_idx.data_ptr(), b, s_q, H, d,
          ratio, topk, P, n_pages, page_size, bits, dt, ws, nbytes)
    return out_idx


def csa_attn_decode_workspace_size(b: int, s_q: int, H: int, d: int, window: int,
                                   cmp_rows: int) -> int:
    """Workspace bytes (0: none needed); cmp_rows = K, or P_cmp * page_size when idx is None.
    Smaller calls may need more (they are cut into more parts), none more than
    2880 * (4 * d + 8) + 16."""
    return int(load_library().csa_attn_decode_workspace_size(b, s_q, H, d, window, cmp_rows))


def csa_attn_decode(q: torch.Tensor, cache: torch.Tensor, raw_table: torch.Tensor,
                    cmp_table: Optional[torch.Tensor], idx: Optional[torch.Tensor],
                    sink: Optional[torch.Tensor], seq_lens: torch.Tensor, scale: float,
                    ratio: int, window: int, page_size: int, bits: int,
                    workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, stream=None
                    ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Sparse MQA of the newest s_q tokens of each sequence over the cache.

    q [b, s_q, H, d], raw_table [b, P_raw] (ring of the raw rows), cmp_table
    [b, P_cmp] (compressed rows; None: window only), idx [b, s_q, K] int32
    (None: every visible block), sink [H] fp32 or None, seq_lens [b] int32.
    Returns (O [b, s_q, H, d], lse [b, s_q, H] fp32).
    """
    if stream is not None and _elsewhere(stream, q):
        return _on(stream, csa_attn_decode, q, cache, raw_table, cmp_table, idx, sink, seq_lens,
                   scale, ratio, window, page_size, bits, workspace, out, lse)
    dev, dt = _first(q, "q", ("b", "s_q", "H", "d"))
    b, s_q, H, d = q.shape
    want = csa_cache_page_bytes(page_size, d, bits)
    n_pages, row = cache.shape if cache.ndim == 2 else (0, -1)
    P_raw = _columns(raw_table, "raw_table")
    if not (row == want and cache.dtype is _U8 and raw_table.dtype is _I32
            and seq_lens.dtype is _I32 and cache.get_device() == dev
            and raw_table.get_device() == dev and seq_lens.get_device() == dev
            and raw_table.shape[0] == b and seq_lens.shape == (b,) and q.is_contiguous()
            and cache.is_contiguous() and raw_table.is_contiguous() and seq_lens.is_contiguous()):
        _refuse(dev, q=(q, q.dtype, q.shape), cache=(cache, _U8, (n_pages, want)),
                raw_table=(raw_table, _I32, (b, P_raw)), seq_lens=(seq_lens, _I32, (b,)))
    P_cmp = K = 0
    cmp_ptr = idx_ptr = sink_ptr = None
    if cmp_table is not None:
        P_cmp = _columns(cmp_table, "cmp_table")
        _optional(cmp_table, "cmp_table", _I32, (b, P_cmp), dev)
        cmp_ptr = cmp_table.data_ptr()
    if idx is not None:
        K = idx.shape[2] if idx.ndim == 3 else 0
        if K == 0 or cmp_table is None:
            raise ValueError("idx needs at least one entry a row, and cmp_table")
        _optional(idx, "idx", _I32, (b, s_q, K), dev)
        idx_ptr = idx.data_ptr()
    if sink is not None:
        _optional(sink, "sink", _F32, (H,), dev)
        sink_ptr = sink.data_ptr()
    if out is None:
        out = _empty((b, s_q, H, d), (s_q * H * d, H * d, d, 1), q.dtype, dev)
    else:
        _optional(out, "out", q.dtype, q.shape, dev)
    if lse is None:
        lse = _empty((b, s_q, H), (s_q * H, H, 1), _F32, dev)
    else:
        _optional(lse, "lse", _F32, (b, s_q, H), dev)
    nbytes = (csa_attn_decode_workspace_size(b, s_q, H, d, window, K or P_cmp * page_size)
              if workspace is None else 0)
    keep, ws, nbytes = _workspace(workspace, nbytes, dev)
    _call("csa_attn_decode", dev, stream, q.data_ptr(), cache.data_ptr(), raw_table.data_ptr(),
          cmp_ptr, idx_ptr, sink_ptr, seq_lens.data_ptr(), float(scale), out.data_ptr(),
          lse.data_ptr(), b, s_q, H, d, ratio, window, K, P_raw, P_cmp, n_pages, page_size, bits,
          dt, ws, nbytes)
    return out, lse
