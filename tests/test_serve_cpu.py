"""The serving calls on the host (no GPU needed): the library exports what
include/csa_serve.h declares, refuses invalid arguments before any CUDA call,
and the binding refuses host tensors and wrong shapes; the oracle of the cache
format is pinned to torch's own conversions."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from compressed_sparse_attention_sum_gb300 import build, csa, serve
from oracle import serve_oracle as orc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "csa_serve.h")
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
FAKE = 0x10000          # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return serve.load_library()


def test_exports_and_signatures(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(csa_[a-z0-9_]+)\s*\(", text))
    assert names == set(serve.SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n


def test_page_bytes(lib):
    assert lib.csa_cache_page_bytes(64, 128, 4) == 64 * (64 + 4)
    assert lib.csa_cache_page_bytes(48, 512, 8) == 48 * (512 + 16)
    for bad in ((64, 128, 5), (8, 128, 4), (24, 128, 4), (64, 48, 4), (64, 544, 4), (64, 0, 4),
                (1 << 17, 128, 4)):
        assert lib.csa_cache_page_bytes(*bad) == 0
        with pytest.raises(ValueError):
            serve.csa_cache_page_bytes(*bad)


def _write(lib, x=FAKE, bs=512, rs=128, dt=1, table=FAKE, pos0=FAKE, counts=None, cache=FAKE, b=1,
           s=4, d=128, P=2, n_pages=4, page=64, bits=4):
    return lib.csa_cache_write(x, bs, rs, dt, table, pos0, counts, cache, b, s, d, P, n_pages, page,
                               bits, None)


def _read(lib, out=FAKE, bs=512, rs=128, dt=1, table=FAKE, pos0=FAKE, counts=None, cache=FAKE, b=1,
          s=4, d=128, P=2, n_pages=4, page=64, bits=4):
    return lib.csa_cache_read(cache, table, pos0, counts, out, bs, rs, dt, b, s, d, P, n_pages, page,
                              bits, None)


@pytest.mark.parametrize("call", [_write, _read])
def test_cache_calls_refuse(lib, call):
    first = {"x": None} if call is _write else {"out": None}
    odd = {k: FAKE + 8 for k in first}
    for bad in (first, odd, dict(table=None), dict(pos0=None), dict(cache=None), dict(cache=FAKE + 4),
                dict(dt=3), dict(bits=3), dict(page=24), dict(d=48), dict(d=544), dict(P=0),
                dict(n_pages=0), dict(b=-1), dict(s=-1), dict(rs=124), dict(rs=64), dict(bs=4),
                dict(P=1 << 26), dict(b=2, bs=-512)):
        assert call(lib, **bad) == INVALID, bad
    assert call(lib, b=70000, bs=0) == UNSUPPORTED
    # nothing to move: accepted without looking at a pointer
    assert call(lib, **first, b=0) == 0 and call(lib, **first, s=0) == 0


def test_read_longer_than_the_ring_is_refused(lib):
    assert _read(lib, s=129, bs=129 * 128) == INVALID


def test_read_into_rows_that_overlap_is_refused(lib):
    for bs in (0, 120):
        assert _read(lib, b=2, bs=bs) == INVALID
    # [s, b, d] rows and a stride that no row uses are not refused for it
    assert _read(lib, b=2, bs=128, rs=256, P=1 << 19) == UNSUPPORTED
    assert _read(lib, bs=0, P=1 << 19) == UNSUPPORTED


def test_infinite_scales_are_refused(lib):
    for x in (float("inf"), -float("inf")):
        assert _attend(lib, scale=x) == INVALID


def _index(lib, q=FAKE, cache=FAKE, table=FAKE, w=FAKE, lens=FAKE, out=FAKE, b=1, s_q=1, H=64, d=128,
           ratio=4, topk=16, P=2, n_pages=4, page=64, bits=4, dt=1, ws=FAKE, nbytes=1 << 30):
    return lib.csa_indexer_topk_decode(q, cache, table, w, lens, out, b, s_q, H, d, ratio, topk, P,
                                       n_pages, page, bits, dt, ws, nbytes, None)


def test_indexer_refuses(lib):
    for k in ("q", "cache", "table", "w", "lens", "out", "ws"):
        assert _index(lib, **{k: None}) == INVALID, k
    for bad in (dict(q=FAKE + 2), dict(cache=FAKE + 8), dict(w=FAKE + 4), dict(ws=FAKE + 8), dict(b=0),
                dict(s_q=0), dict(H=0), dict(ratio=0), dict(topk=0), dict(P=0), dict(n_pages=0),
                dict(bits=2), dict(page=17), dict(d=40), dict(dt=9)):
        assert _index(lib, **bad) == INVALID, bad
    for bad in (dict(d=288), dict(H=129), dict(b=40000, s_q=2), dict(P=1 << 19)):
        assert _index(lib, **bad) == UNSUPPORTED, bad
    need = lib.csa_indexer_topk_decode_workspace_size(1, 1, 64, 128, 128)
    assert need > 0 and _index(lib, nbytes=need - 1) == WORKSPACE
    assert lib.csa_indexer_topk_decode_workspace_size(0, 1, 64, 128, 128) == 0


def _attend(lib, q=FAKE, cache=FAKE, raw=FAKE, cmp=FAKE, idx=FAKE, sink=None, lens=FAKE, scale=0.1,
            o=FAKE, lse=FAKE, b=1, s_q=1, H=32, d=128, ratio=4, window=64, K=256, P_raw=2, P_cmp=8,
            n_pages=16, page=64, bits=4, dt=1, ws=FAKE, nbytes=1 << 30):
    return lib.csa_attn_decode(q, cache, raw, cmp, idx, sink, lens, scale, o, lse, b, s_q, H, d, ratio,
                               window, K, P_raw, P_cmp, n_pages, page, bits, dt, ws, nbytes, None)


def test_attention_refuses(lib):
    for k in ("q", "cache", "raw", "cmp", "lens", "o", "lse"):
        assert _attend(lib, **{k: None}) == INVALID, k
    for bad in (dict(q=FAKE + 2), dict(cache=FAKE + 8), dict(o=FAKE + 4), dict(ws=FAKE + 8), dict(b=0),
                dict(s_q=0), dict(H=0), dict(ratio=0), dict(window=0), dict(K=-1), dict(K=0),
                dict(idx=None), dict(P_raw=0), dict(P_cmp=-1), dict(P_cmp=0), dict(n_pages=0),
                dict(bits=6), dict(page=8), dict(d=100), dict(dt=2), dict(scale=float("nan")),
                dict(window=129), dict(window=128, s_q=2)):
        assert _attend(lib, **bad) == INVALID, bad
    for bad in (dict(H=129), dict(b=65536), dict(K=(1 << 24) + 1), dict(idx=None, K=0, P_cmp=1 << 19)):
        assert _attend(lib, **bad) == UNSUPPORTED, bad
    need = lib.csa_attn_decode_workspace_size(1, 1, 32, 128, 64, 256)
    assert need > 0                                    # one query: its slots are split
    assert _attend(lib, nbytes=need - 1) == WORKSPACE
    assert _attend(lib, ws=None) == WORKSPACE


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


I32, U8, F32 = torch.int32, torch.uint8, torch.float32
CALLS = {
    "csa_cache_write": lambda: serve.csa_cache_write(
        _t(1, 4, 32), _t(2, 288, dtype=U8), _t(1, 2, dtype=I32), _t(1, dtype=I32), 16, 4),
    "csa_cache_read": lambda: serve.csa_cache_read(
        _t(2, 288, dtype=U8), _t(1, 2, dtype=I32), _t(1, dtype=I32), _t(1, 4, 32), 16, 4),
    "csa_indexer_topk_decode": lambda: serve.csa_indexer_topk_decode(
        _t(1, 1, 2, 32), _t(2, 288, dtype=U8), _t(1, 2, dtype=I32), _t(1, 1, 2, dtype=F32),
        _t(1, dtype=I32), 2, 4, 16, 4),
    "csa_attn_decode": lambda: serve.csa_attn_decode(
        _t(1, 1, 2, 32), _t(2, 288, dtype=U8), _t(1, 1, dtype=I32), None, None, None,
        _t(1, dtype=I32), 0.1, 4, 8, 16, 4),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_host_tensors_are_rejected(name):
    with pytest.raises(ValueError, match="CUDA tensor"):
        CALLS[name]()


def test_every_compute_call_is_covered():
    assert {n for n in serve.SIGNATURES if not n.endswith(("_size", "_bytes"))} == set(CALLS)


def test_binding_fails_loudly_without_library(tmp_path, monkeypatch):
    monkeypatch.setattr(csa, "_lib", None)
    monkeypatch.setattr(csa.load_library, "__defaults__", (str(tmp_path / "missing.so"),))
    with pytest.raises(RuntimeError):
        serve.load_library()


# ------------------------------------------------------------- oracle pins

def test_e4m3_codes_match_torch():
    g = np.random.default_rng(0)
    x = np.concatenate([g.standard_normal(4000), g.standard_normal(2000) * 1e-3,
                        np.array([0.0, -0.0, 448.0, 1.0, 1.0625, 1.1875, 2 ** -9, 2 ** -10, 3 * 2 ** -10])])
    x = np.resize(x, 6016).reshape(-1, 32)
    x[:, 0] = 448.0                                    # every group's exponent is 0
    x = x.astype(np.float32).astype(np.float64)
    codes, exps = orc.quantize_rows(x, 8)
    assert (exps == 0).all()
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn)
    assert np.array_equal(codes, want.view(torch.uint8).numpy())
    assert np.array_equal(orc.code_values(codes, exps, 8), want.double().numpy())


def test_e2m1_rounding_by_hand():
    pairs = [(0.2, 0), (0.25, 0), (0.26, .5), (0.75, 1), (0.74, .5), (1.25, 1), (1.75, 2), (2.5, 2),
             (2.51, 3), (3.5, 4), (5.0, 4), (5.01, 6), (6.0, 6)]
    x = np.zeros(32)
    x[:13] = [p[0] for p in pairs]
    x[13:26] = [-p[0] for p in pairs]
    got = orc.held_rows(x[None], 4)[0]
    assert np.array_equal(got[:13], [p[1] for p in pairs])
    assert np.array_equal(got[13:26], [-p[1] for p in pairs])


@pytest.mark.parametrize("bits,top", [(4, 6.0), (8, 448.0)])
def test_exponent_is_the_smallest_that_holds(bits, top):
    for amax, want in ((top, 0), (np.nextafter(np.float32(top), np.float32(1e9)), 1), (top / 2, -1),
                       (2 * top, 1), (0.0, -110), (1e-38, -110)):
        x = np.zeros((1, 32))
        x[0, 5] = -amax
        assert orc.quantize_rows(x, bits)[1][0, 0] == want, amax


def test_held_rows_are_bf16_values_within_half_a_step():
    x = np.random.default_rng(1).standard_normal((3, 64))
    # half the widest step is 2^e (4 to 6) of e2m1 and 16 * 2^e (416 to 448) of e4m3, and the group's
    # largest magnitude is above 3 * 2^e, 224 * 2^e (a smaller exponent would hold it otherwise)
    for bits, rel in ((4, 1.0 / 3), (8, 1.0 / 14)):
        v = orc.held_rows(x, bits)
        t = torch.from_numpy(v)
        assert torch.equal(t.bfloat16().double(), t)
        amax = np.abs(x).reshape(3, 2, 32).max(-1).repeat(32, -1)
        assert (np.abs(v - x) <= rel * amax).all()


def test_attend_row_against_torch_softmax():
    g = torch.Generator().manual_seed(3)
    q = torch.randn(3, 8, generator=g, dtype=torch.float64)
    raw = torch.randn(12, 8, generator=g, dtype=torch.float64)
    cmp = torch.randn(4, 8, generator=g, dtype=torch.float64)
    sink = torch.randn(3, generator=g, dtype=torch.float64)
    o, lse, _ = orc.attend_row(q.numpy(), lambda p: raw[p].numpy(), lambda j: cmp[j].numpy(),
                               [2, -1, 0, 2, 3], sink.numpy(), 0.3, 11, 4, 5)
    kv = torch.cat([raw[7:12], cmp[2:3], cmp[0:1], cmp[2:3]])       # block 3 is not visible yet
    z = torch.cat([q @ kv.T * 0.3, sink[:, None]], 1)
    assert np.allclose(o, (torch.softmax(z, 1)[:, :-1] @ kv).numpy(), atol=1e-13)
    assert np.allclose(lse, torch.logsumexp(z, 1).numpy(), atol=1e-13)
