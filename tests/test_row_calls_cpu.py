"""The row calls and csa_compress_decode on the host (no GPU needed): the library
exports what include/csa_rows.h declares, refuses invalid arguments before any CUDA
call, the binding refuses host tensors; frequencies and turns against their formulas;
the oracle against torch's autograd."""
import ctypes
import glob
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from compressed_sparse_attention_sum_gb300 import build, csa, rows
from oracle import rows_oracle as orc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "csa_rows.h")
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
FAKE = 0x10000          # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return rows.load_library()


def test_exports_and_signatures(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(csa_[a-z0-9_]+)\s*\(", text))
    assert names == set(rows.SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n


def strides(batch=0, token=0, head=0):
    return ctypes.byref(rows._Strides(batch, token, head))


def plan(turns=FAKE, dim=64, first=64, layout=0, scale=1.0):
    return ctypes.byref(rows._RopeStruct(turns, dim, first, layout, scale))


def _norm(lib, x=FAKE, xs=4096, dt=1, kind=1, weight=FAKE, bias=None, eps=1e-6, out=FAKE, os=4096, n_rows=4, n=4096):
    return lib.csa_norm(x, xs, dt, kind, weight, bias, eps, out, os, n_rows, n, None)


def _norm_bwd(lib, x=FAKE, xs=4096, dt=1, kind=1, weight=FAKE, eps=1e-6, dout=FAKE, gs=4096, g_dt=1, dx=FAKE, ds=4096, dx_dt=1,
              dweight=FAKE, dbias=None, n_rows=4, n=4096, ws=FAKE, nbytes=1 << 30):
    return lib.csa_norm_bwd(x, xs, dt, kind, weight, eps, dout, gs, g_dt, dx, ds, dx_dt, dweight, dbias, n_rows, n, ws, nbytes, None)


def test_norm_refuses(lib):
    for bad in (dict(x=None), dict(out=None), dict(x=FAKE + 8), dict(out=FAKE + 2), dict(weight=FAKE + 4), dict(bias=FAKE + 8),
                dict(dt=2), dict(kind=0), dict(kind=3), dict(eps=-1.0), dict(eps=float("inf")), dict(eps=float("nan")), dict(n=4092),
                dict(n=0), dict(n_rows=-1), dict(xs=4100), dict(xs=-4096), dict(os=4088), dict(os=0), dict(os=4100)):
        assert _norm(lib, **bad) == INVALID, bad
    assert _norm(lib, n=32776, os=32776) == UNSUPPORTED
    assert _norm(lib, n_rows=1 << 31) == UNSUPPORTED
    assert _norm(lib, x=None, out=None, n_rows=0) == 0


def test_norm_bwd_refuses(lib):
    for bad in (dict(x=None), dict(dout=None), dict(dx=None), dict(dout=FAKE + 8), dict(dx=FAKE + 8), dict(dweight=FAKE + 4),
                dict(dbias=FAKE + 4), dict(ws=FAKE + 8), dict(g_dt=7), dict(dx_dt=-1), dict(kind=0), dict(gs=4092), dict(ds=4000),
                dict(eps=-0.5), dict(n=12)):
        assert _norm_bwd(lib, **bad) == INVALID, bad
    assert _norm_bwd(lib, n=40000, xs=40000, gs=40000, ds=40000) == UNSUPPORTED
    need = lib.csa_norm_bwd_workspace_size(4, 4096, 1, 0)
    assert need > 0 and _norm_bwd(lib, nbytes=need - 1) == WORKSPACE and _norm_bwd(lib, ws=None) == WORKSPACE
    assert lib.csa_norm_bwd_workspace_size(4, 4096, 0, 0) == 0 == lib.csa_norm_bwd_workspace_size(0, 4096, 1, 1)
    assert lib.csa_norm_bwd_workspace_size(4, 4096, 1, 1) == 2 * need
    # no rows: nothing but the sums, which are not wanted here, is looked at
    assert _norm_bwd(lib, x=None, dout=None, dx=None, dweight=None, ws=None, n_rows=0) == 0


def _rope(lib, x=FAKE, xs=(65536, 4096, 128), dt=1, pos=None, ps=0, rope=None, inverse=0, out=FAKE, os=(65536, 4096, 128), b=2, s=16,
          H=32, d=128, call="csa_rope"):
    rope = plan() if rope is None else rope
    if call == "csa_rope":
        return lib.csa_rope(x, strides(*xs), dt, pos, ps, rope, inverse, out, strides(*os), b, s, H, d, None)
    if call == "csa_rope_bwd":
        return lib.csa_rope_bwd(x, strides(*xs), dt, pos, ps, rope, inverse, out, strides(*os), dt, b, s, H, d, None)
    if call == "csa_norm_rope":
        return lib.csa_norm_rope(x, strides(*xs), dt, 1, FAKE, None, 1e-6, pos, ps, rope, out, strides(*os), b, s, H, d, None)
    return lib.csa_norm_rope_bwd(x, strides(*xs), dt, 1, FAKE, 1e-6, pos, ps, rope, FAKE, strides(*xs), 0, out, strides(*os), dt, FAKE,
                                 None, b, s, H, d, FAKE, 1 << 30, None)


CALLS = ["csa_rope", "csa_rope_bwd", "csa_norm_rope", "csa_norm_rope_bwd"]


@pytest.mark.parametrize("call", CALLS)
def test_rope_calls_refuse(lib, call):
    for bad in (dict(x=None), dict(out=None), dict(x=FAKE + 4), dict(out=FAKE + 8), dict(dt=5), dict(b=-1), dict(s=-1), dict(H=-1),
                dict(d=132), dict(d=0), dict(pos=FAKE + 2), dict(pos=FAKE, ps=-1), dict(xs=(65536, 4100, 128)),
                dict(xs=(-65536, 4096, 128)), dict(os=(65536, 4096, 120)), dict(os=(65536, 4088, 128)), dict(os=(65536, 0, 128)),
                dict(os=(4096, 4096, 128)), dict(os=(61440, 4096, 128)), dict(os=(61440 + 64, 4096, 128))):
        assert _rope(lib, **bad, call=call) == INVALID, bad
    for bad in (dict(turns=None), dict(turns=FAKE + 8), dict(dim=0), dict(dim=63), dict(dim=130, first=0), dict(first=66), dict(first=-2),
                dict(first=63), dict(layout=2), dict(layout=1, dim=62), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _rope(lib, rope=plan(**bad), call=call) == INVALID, bad
    # strides that no two rows use do not matter
    assert _rope(lib, d=520, H=1, os=(1 << 20, 1 << 12, 0), call=call) == UNSUPPORTED
    assert _rope(lib, b=1 << 12, s=1 << 12, H=1 << 8, xs=(0, 0, 0), os=(1 << 40, 1 << 20, 128), call=call) == UNSUPPORTED
    assert _rope(lib, x=None, out=None, b=0, call=call) == 0 or call == "csa_norm_rope_bwd"


def test_rows_in_any_order_of_strides_are_taken(lib):
    """[H, s, b, d] in memory: not refused for its strides (d is beyond the limit)."""
    assert _rope(lib, b=2, s=16, H=32, d=520, os=(520, 1040, 1040 * 16)) == UNSUPPORTED
    assert _rope(lib, b=2, s=16, H=32, d=520, os=(520, 1040, 1040 * 16 - 8)) == INVALID


def _compress(lib, kv=FAKE, kb=512, kr=128, score=FAKE, sb=512, sr=128, sw=128, kv_ring=FAKE, score_ring=FAKE, R=16, lens=FAKE, kind=1,
              weight=FAKE, bias=None, eps=1e-6, rope="default", out=FAKE, ob=256, first=FAKE, counts=FAKE, b=2, s_q=4, d=128, ratio=4,
              coff=2, dt=1):
    rope = plan() if rope == "default" else rope
    return lib.csa_compress_decode(kv, kb, kr, score, sb, sr, sw, kv_ring, score_ring, R, lens, kind, weight, bias, eps, rope, out, ob,
                                   first, counts, b, s_q, d, ratio, coff, dt, None)


def test_compress_decode_refuses(lib):
    for k in ("kv", "score", "kv_ring", "score_ring", "lens", "out", "first", "counts"):
        assert _compress(lib, **{k: None}) == INVALID, k
    for bad in (dict(kv=FAKE + 8), dict(score=FAKE + 8), dict(kv_ring=FAKE + 8), dict(score_ring=FAKE + 8), dict(out=FAKE + 8),
                dict(kr=124), dict(kr=-128), dict(kb=-512), dict(kb=500), dict(sr=100), dict(sb=-512), dict(sw=2), dict(R=7), dict(kind=3),
                dict(kind=-1), dict(weight=FAKE + 4), dict(eps=-1.0), dict(rope=plan(dim=63)), dict(ob=120), dict(ob=260),
                dict(d=124), dict(ratio=0), dict(coff=0), dict(b=-1), dict(s_q=-1), dict(dt=3), dict(sw=1, score=FAKE + 1),
                dict(sw=1, sr=-1)):
        assert _compress(lib, **bad) == INVALID, bad
    for bad in (dict(d=520, kr=520, kb=4160, sw=1, ob=520), dict(coff=3), dict(b=65536), dict(R=(1 << 24) + 1)):
        assert _compress(lib, **bad) == UNSUPPORTED, bad
    assert _compress(lib, kv=None, b=0) == 0 and _compress(lib, kv=None, s_q=0) == 0


def test_frequencies_and_turns(lib):
    for args in ((64,), (64, 40000.0), (2, 10000.0), (22, 500.0, "linear", 4.0), (128, 10000.0, "by_parts", 16.0, 4096.0),
                 (64, 10000.0, "by_parts", 40.0, 4096.0, 16.0, 2.0), (64, 1e6, "by_parts", 8.0, 64.0)):
        got, want = rows.csa_rope_freqs(*args).numpy(), orc.freqs(*args)
        assert np.abs(got - want).max() <= 1e-15 * np.abs(want).max() + 4 * 2.0 ** -53 * np.abs(want).max(), args
        turns = rows.csa_rope_turns(got, "cpu").numpy().astype(np.uint64).astype(np.float64) * 2.0 ** -64
        # one division, one conversion
        assert np.abs(turns - got / (2 * np.pi)).max() <= 2.0 ** -52
    # whole turns drop out; a frequency may be negative
    t = rows.csa_rope_turns([2 * np.pi * 3, -np.pi / 2, 0.0], "cpu").tolist()
    assert abs((t[0] + (1 << 63)) % (1 << 64) - (1 << 63)) <= 1 << 14 and abs(t[1] % (1 << 64) - 3 * (1 << 62)) <= 1 << 12 and t[2] == 0
    out = (ctypes.c_double * 8)()
    for bad in ((3, 1e4, 0, 1.0, 0.0, 32.0, 1.0), (0, 1e4, 0, 1.0, 0.0, 32.0, 1.0), (8, 0.0, 0, 1.0, 0.0, 32.0, 1.0),
                (8, 1e4, 1, 0.0, 0.0, 32.0, 1.0), (8, 1e4, 2, 4.0, 0.0, 32.0, 1.0), (8, 1.0, 2, 4.0, 64.0, 32.0, 1.0),
                (8, 1e4, 2, 4.0, 64.0, 1.0, 2.0), (8, 1e4, 3, 4.0, 64.0, 32.0, 1.0), (8, float("inf"), 0, 1.0, 0.0, 32.0, 1.0)):
        assert lib.csa_rope_freqs(*bad, out) == INVALID, bad
    with pytest.raises(csa.CSAError):
        rows.csa_rope_turns([float("nan")], "cpu")
    with pytest.raises(csa.CSAError):
        rows.csa_rope_turns([], "cpu")


def test_host_tensors_are_refused():
    z = torch.zeros(1, 4, 8, dtype=torch.bfloat16)
    lens = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: rows.csa_norm(z, 1), lambda: rows.csa_norm_bwd(z, z, 1), lambda: rows.csa_rope(z, None),
                 lambda: rows.csa_rope_bwd(z, None), lambda: rows.csa_norm_rope(z, 1, None),
                 lambda: rows.csa_norm_rope_bwd(z, z, 1, None), lambda: rows.CsaRope(torch.zeros(4, dtype=torch.int64)),
                 lambda: rows.csa_compress_decode(z, z, z, z, lens, 4)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.mark.parametrize("kind", [orc.RMS, orc.LAYER])
@pytest.mark.parametrize("half", [False, True])
def test_oracle_gradients_are_those_of_autograd(kind, half):
    rng = np.random.default_rng(5)
    x, dy, w, b = rng.standard_normal((6, 24)), rng.standard_normal((6, 24)), rng.standard_normal(24), rng.standard_normal(24)
    f, pos = orc.freqs(16), np.array([0, 1, 5, -3, 100000, 7])
    tx, tw, tb = (torch.tensor(t, requires_grad=True) for t in (x, w, b))
    m = tx.mean(-1, keepdim=True) if kind == orc.LAYER else 0
    y = (tx - m) / torch.sqrt(((tx - m) ** 2).mean(-1, keepdim=True) + 1e-5) * tw + tb
    u, v = (torch.tensor(i) for i in orc.pairs(16, 8, half))
    a = torch.tensor(pos)[:, None] * torch.tensor(f)
    z = y.clone()
    z[:, u] = 1.5 * (y[:, u] * a.cos() - y[:, v] * a.sin())
    z[:, v] = 1.5 * (y[:, u] * a.sin() + y[:, v] * a.cos())
    want = torch.autograd.grad(z, (tx, tw, tb), torch.tensor(dy))
    fwd, _ = orc.turn(orc.norm(x, kind, w, b, 1e-5)[0], pos, f, 8, half, 1.5)
    assert np.abs(fwd - z.detach().numpy()).max() < 1e-12
    back, e = orc.turn(dy, pos, f, 8, half, 1.5, back=True)
    got, _ = orc.norm_bwd(x, back, e, kind, w, 1e-5)
    for g, t in zip(got, want):
        assert np.abs(g - t.numpy()).max() < 1e-11


def test_gradients_without_rows_look_at_no_pointer_but_the_sums(lib):
    """... and at none where these are not wanted; misaligned ones are refused before they are written."""
    def call(dweight, dbias, **size):
        at = dict(dict(b=2, s=16, H=32), **size)
        return lib.csa_norm_rope_bwd(None, None, 1, 1, None, 1e-6, None, 0, None, None, None, 0, None, None, 1, dweight, dbias, at["b"],
                                     at["s"], at["H"], 128, None, 0, None)
    for none in (dict(b=0), dict(s=0), dict(H=0)):
        assert call(None, None, **none) == 0
        assert call(FAKE + 4, None, **none) == call(None, FAKE + 8, **none) == INVALID
    assert call(None, None) == INVALID


def test_made_up_addresses_meet_no_gpu(request):
    """The one test whose made-up address a kernel would write to is skipped where there is a GPU."""
    import conftest
    assert conftest.HOST_ONLY == ("test_row_calls_cpu.py::test_rope_calls_refuse[csa_norm_rope_bwd]",)
    item = [i for i in request.session.items if i.nodeid.endswith(conftest.HOST_ONLY)]
    assert all([m.args for m in i.iter_markers("skipif")] == [("__import__('torch').cuda.is_available()",)] for i in item)


def test_numbers_beyond_32_bits_are_not_cut(lib):
    """2^32 more than a size that a call takes: nothing of it may count as the small size."""
    far = 2 ** 32
    for dim in (64 + far, 64 - far, 2 ** 31):
        with pytest.raises(ValueError, match="2\\^31"):
            rows.csa_rope_freqs(dim)
    with pytest.raises(ValueError, match="2\\^31"):
        rows.csa_rope_turns(torch.zeros(1, dtype=torch.float64).expand(1 + far), "cpu")
    for kind in (1 + far, 2 + far, 1 - far, far, -1, 4):
        with pytest.raises(ValueError, match="kind"):
            rows._kind(kind)
    assert [rows._kind(k) for k in (0, 1, 2, 3)] == [0, 1, 2, 3]


def test_angles_are_products_modulo_a_turn(tmp_path):
    """The kernels' angle against whole numbers of any size, as constant expressions: those may not overflow."""
    top = 2 ** 31
    cases = [(t, p) for t in (0, 1, 2 ** 62 + 12345, 2 ** 63 - 1, -1, -2 ** 63 + 1, -2 ** 63, 0x123456789abcdef) for p in (0, 1, -1, 3, 1 << 20, top - 1, -top)]
    lines = [f"static_assert(csa::angle_of((int64_t){t % 2 ** 64}ull, {p if p > -top else '-2147483647 - 1'}) == {t * p % 2 ** 64 >> 32}u, \"\");"
             for t, p in cases]
    src = tmp_path / "angles.cpp"
    src.write_text('#include "rows.h"\n' + "\n".join(lines) + "\n")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    r = subprocess.run(["g++", "-std=c++17", "-fsyntax-only", "-I", build.CSRC, "-I", cuda, "-I", "/usr/local/cuda/include", str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]


def test_dependent_kernels_read_what_their_predecessor_wrote():
    """A row call's kernel that starts before its predecessor's end and waits for it: its pointers are not __restrict__, of which a
    const one may be read through the cache of data that no kernel writes meanwhile, and before the wait."""
    seen = set()
    for path in glob.glob(os.path.join(build.CSRC, "rows_*.cu")):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        starts = [m.start() for m in re.finditer(r"__global__", src)] + [len(src)]
        for a, b in zip(starts, starts[1:]):
            if "griddepcontrol.wait" in src[a:b]:
                head = src[a:src.index("{", a)]
                seen.add(re.search(r"(\w+_kernel)\(", head).group(1))
                assert "__restrict__" not in head, (os.path.basename(path), head)
    assert seen == {"sum_parts_kernel"}
