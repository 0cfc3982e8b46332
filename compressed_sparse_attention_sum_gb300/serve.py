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
from .csa import CSAError, _dt, _need, _ptr  # noqa: F401  (CSAError: re-exported)

_c_int, _c_ll, _c_p, _c_f, _c_sz = (ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p,
                                    ctypes.c_float, ctypes.c_size_t)

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


def _same_device(first: torch.Tensor, **others):
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, expected {first.device}")


def _call(name: str, t: torch.Tensor, stream, *args):
    """Call an entry point with t's device current, on `stream` or on that device's current one."""
    lib = load_library()
    with torch.cuda.device(t.device):
        s = stream if stream is not None else torch.cuda.current_stream(t.device)
        csa._check(name, getattr(lib, name)(*args, s.cuda_stream))


def _cache_args(cache, page_size, bits, d):
    """Check the cache tensor [n_pages, page bytes] and return n_pages."""
    _need(cache, "cache", dtype=torch.uint8)
    want = csa_cache_page_bytes(page_size, d, bits)
    if cache.dim() != 2 or cache.shape[1] != want:
        raise ValueError(f"cache must be [n_pages, {want}] for pages of {page_size} rows of {d} "
                         f"channels in {bits} bits, got {tuple(cache.shape)}")
    return cache.shape[0]


def _int_tensor(t, name, shape, optional=False):
    if t is None and optional:
        return
    _need(t, name, dtype=torch.int32)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _table(t, name, b):
    _need(t, name, dtype=torch.int32)
    if t.dim() != 2 or t.shape[0] != b or t.shape[1] < 1:
        raise ValueError(f"{name} must be [{b}, P] with P >= 1, got {tuple(t.shape)}")
    return t.shape[1]


def _workspace(ws, nbytes, dev):
    if ws is None:
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    _need(ws, "workspace")
    return ws


def csa_cache_page_bytes(page_size: int, d: int, bits: int) -> int:
    """Bytes of one page of `page_size` rows of d channels in 4 or 8 bits."""
    n = int(load_library().csa_cache_page_bytes(int(page_size), int(d), int(bits)))
    if n == 0:
        raise ValueError(f"no cache format with pages of {page_size} rows, {d} channels and "
                         f"{bits} bits (page_size % 16 == 0, d % 32 == 0, d <= 512, bits 4 or 8)")
    return n


def _rows_args(x, name, cache, table, pos0, page_size, bits, counts):
    _need(x, name, contiguous=False)
    if x.dim() != 3:
        raise ValueError(f"{name} must be [b, s, d]")
    b, s, d = x.shape
    if x.numel() and x.stride(2) != 1:
        raise ValueError(f"{name} rows must be contiguous")
    n_pages = _cache_args(cache, page_size, bits, d)
    P = _table(table, "table", b) if b else 1
    _int_tensor(pos0, "pos0", (b,))
    _int_tensor(counts, "counts", (b,), optional=True)
    _same_device(x, cache=cache, table=table, pos0=pos0, counts=counts)
    return b, s, d, P, n_pages


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
    b, s, d, P, n_pages = _rows_args(x, "x", cache, table, pos0, page_size, bits, counts)
    if b and s:
        _call("csa_cache_write", x, stream, x.data_ptr(), x.stride(0), x.stride(1), _dt(x),
              table.data_ptr(), pos0.data_ptr(), _ptr(counts), cache.data_ptr(), b, s, d, P,
              n_pages, page_size, bits)
    return cache


def csa_cache_read(cache: torch.Tensor, table: torch.Tensor, pos0: torch.Tensor,
                   out: torch.Tensor, page_size: int, bits: int,
                   counts: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Read the rows at positions pos0[s] .. pos0[s] + counts[s] - 1 into
    out [b, s, d] (bf16 or fp32, rows contiguous), exactly as the codes stand
    for them; rows past counts[s] are left as they were.  Returns out."""
    b, s, d, P, n_pages = _rows_args(out, "out", cache, table, pos0, page_size, bits, counts)
    if b and s:
        _call("csa_cache_read", out, stream, cache.data_ptr(), table.data_ptr(), pos0.data_ptr(),
              _ptr(counts), out.data_ptr(), out.stride(0), out.stride(1), _dt(out), b, s, d, P,
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
    _need(q_I, "q_I")
    if q_I.dim() != 4:
        raise ValueError("q_I must be [b, s_q, H_I, d_I]")
    b, s_q, H, d = q_I.shape
    n_pages = _cache_args(cache, page_size, bits, d)
    P = _table(table, "table", b)
    _need(w, "w", dtype=torch.float32)
    if tuple(w.shape) != (b, s_q, H):
        raise ValueError(f"w must be {(b, s_q, H)}, got {tuple(w.shape)}")
    _int_tensor(seq_lens, "seq_lens", (b,))
    if out_idx is None:
        out_idx = torch.empty(b, s_q, max(topk, 0), dtype=torch.int32, device=q_I.device)
    _int_tensor(out_idx, "out_idx", (b, s_q, topk))
    if workspace is None:
        nbytes = csa_indexer_topk_decode_workspace_size(b, s_q, H, d, P * page_size)
        workspace = _workspace(None, nbytes, q_I.device)
    _need(workspace, "workspace")
    _same_device(q_I, cache=cache, table=table, w=w, seq_lens=seq_lens, out_idx=out_idx,
                 workspace=workspace)
    _call("csa_indexer_topk_decode", q_I, stream, q_I.data_ptr(), cache.data_ptr(),
          table.data_ptr(), w.data_ptr(), seq_lens.data_ptr(), out_idx.data_ptr(), b, s_q, H, d,
          ratio, topk, P, n_pages, page_size, bits, _dt(q_I), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return out_idx


def csa_attn_decode_workspace_size(b: int, s_q: int, H: int, d: int, window: int,
                                   cmp_rows: int) -> int:
    """Workspace bytes (0: none needed); cmp_rows = K, or P_cmp * page_size when idx is None."""
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
    _need(q, "q")
    if q.dim() != 4:
        raise ValueError("q must be [b, s_q, H, d]")
    b, s_q, H, d = q.shape
    n_pages = _cache_args(cache, page_size, bits, d)
    P_raw = _table(raw_table, "raw_table", b)
    P_cmp = 0 if cmp_table is None else _table(cmp_table, "cmp_table", b)
    K = 0
    if idx is not None:
        _need(idx, "idx", dtype=torch.int32)
        if idx.dim() != 3 or tuple(idx.shape[:2]) != (b, s_q):
            raise ValueError(f"idx must be [{b}, {s_q}, K], got {tuple(idx.shape)}")
        K = idx.shape[2]
        if K == 0 or cmp_table is None:
            raise ValueError("idx needs at least one entry a row, and cmp_table")
    if sink is not None:
        _need(sink, "sink", dtype=torch.float32)
        if tuple(sink.shape) != (H,):
            raise ValueError(f"sink must be [{H}]")
    _int_tensor(seq_lens, "seq_lens", (b,))
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(b, s_q, H, dtype=torch.float32, device=q.device)
    _need(out, "out", dtype=q.dtype)
    _need(lse, "lse", dtype=torch.float32)
    if out.shape != q.shape or tuple(lse.shape) != (b, s_q, H):
        raise ValueError("out must have q's shape and lse [b, s_q, H]")
    if workspace is None:
        nbytes = csa_attn_decode_workspace_size(b, s_q, H, d, window, K or P_cmp * page_size)
        workspace = _workspace(None, nbytes, q.device)
    _need(workspace, "workspace")
    _same_device(q, cache=cache, raw_table=raw_table, cmp_table=cmp_table, idx=idx, sink=sink,
                 seq_lens=seq_lens, out=out, lse=lse, workspace=workspace)
    _call("csa_attn_decode", q, stream, q.data_ptr(), cache.data_ptr(), raw_table.data_ptr(),
          _ptr(cmp_table), _ptr(idx), _ptr(sink), seq_lens.data_ptr(), float(scale),
          out.data_ptr(), lse.data_ptr(), b, s_q, H, d, ratio, window, K, P_raw, P_cmp, n_pages,
          page_size, bits, _dt(q), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return out, lse
