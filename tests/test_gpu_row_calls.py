"""The row calls on the GPU against the fp64 oracle (oracle/rows_oracle.py, which also
derives how far fp32 arithmetic may be off): norms, rotary positions and both in one
pass, their gradients, strides, types, positions, streams and graphs."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from compressed_sparse_attention_sum_gb300 import csa, rows
from oracle import rows_oracle as orc

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
NAME = {BF: "bf16", F32: "fp32"}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from compressed_sparse_attention_sum_gb300 import build
    build.build()
    rows.load_library()
    csa.csa_get_device_status()
    yield
    assert csa.csa_get_device_status() == 0


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def draw(rng, *shape, dtype=F32, shift=0.0):
    """Channels of different size and mean, as a tensor on the GPU and in fp64."""
    x = rng.standard_normal(shape) * np.exp(0.5 * rng.standard_normal(shape[-1])) + shift
    t = torch.tensor(x, dtype=F32).to(dtype).cuda()
    return t, f64(t)


def close(got, want, err, what=""):
    """got within err of want and half a step of its type."""
    g = f64(got)
    bound = err + orc.STEP[NAME[got.dtype]] * (np.abs(want) + err) + 1e-37
    assert g.shape == want.shape
    off = np.abs(g - want) / bound
    assert np.isfinite(g).all() and off.max(initial=0) <= 1, (what, float(off.max()), np.unravel_index(off.argmax(), off.shape))


def plan(f, first, half, scale=1.0):
    return rows.CsaRope(rows.csa_rope_turns(f), first, "half" if half else "interleaved", scale)


# ------------------------------------------------------------------- norms

WIDTHS = [8, 16, 24, 40, 64, 128, 136, 200, 256, 504, 512, 520, 1000, 1024, 2056, 4096, 4104, 7168, 8192, 8200, 16384, 16392, 32768]


@pytest.mark.parametrize("kind", [orc.RMS, orc.LAYER])
@pytest.mark.parametrize("n", WIDTHS)
def test_norm_and_its_gradient(n, kind):
    rng = np.random.default_rng(n + kind)
    for r, dtype, g_dt, dx_dt in ((1, BF, BF, BF), (7, F32, F32, F32), (67 if n < 5000 else 33, BF, F32, F32), (19, F32, BF, BF)):
        x, x64 = draw(rng, r, n, dtype=dtype, shift=0.5)
        dy, dy64 = draw(rng, r, n, dtype=g_dt)
        w, w64 = draw(rng, n)
        b, b64 = draw(rng, n)
        for weight, bias in ((True, True), (True, False), (False, False)):
            ww, bb = (w64 if weight else None), (b64 if bias else None)
            out = rows.csa_norm(x, kind, w if weight else None, b if bias else None, EPS)
            close(out, *orc.norm(x64, kind, ww, bb, EPS), what=("norm", n, r, dtype))
            dx = torch.empty(r, n, dtype=dx_dt, device="cuda")
            got = rows.csa_norm_bwd(x, dy, kind, w if weight else None, EPS, has_bias=bias, dx=dx)
            want, err = orc.norm_bwd(x64, dy64, 0 * dy64, kind, ww, EPS)
            assert got[0] is dx and (got[1] is None) == (not weight) and (got[2] is None) == (not bias)
            for k, t in enumerate(got):
                if t is not None:
                    close(t, want[k], err[k], what=("norm_bwd", k, n, r, dtype))


@pytest.mark.parametrize("n", [128, 4096])
def test_gradient_against_differences(n):
    """fp32: dx and dweight along a direction against the forward call's differences, in the oracle's bounds
    of the two forward results and the second derivative's share."""
    rng = np.random.default_rng(3)
    x, _ = draw(rng, 4, n)
    v, _ = draw(rng, 4, n)
    dy, dy64 = draw(rng, 4, n)
    w, w64 = draw(rng, n)
    h = 2.0 ** -6
    for kind in (orc.RMS, orc.LAYER):
        dx, dw, _ = rows.csa_norm_bwd(x, dy, kind, w, EPS)
        hi, lo = x + h * v, x - h * v
        v64 = (f64(hi) - f64(lo)) / (2 * h)             # the step that fp32 took
        (yh, eh), (yl, el) = (orc.norm(f64(t), kind, w64, None, EPS) for t in (hi, lo))
        gh, gl = (f64(rows.csa_norm(t, kind, w, None, EPS)) for t in (hi, lo))
        slope = ((gh - gl) * dy64).sum() / (2 * h)
        exact = ((yh - yl) * dy64).sum() / (2 * h)
        tell = (f64(dx) * v64).sum()
        fwd_err = ((eh + el + orc.STEP["fp32"] * (np.abs(yh) + np.abs(yl))) * np.abs(dy64)).sum() / (2 * h)
        assert abs(slope - exact) <= fwd_err
        # the central difference's own error: h^2 / 6 times the third derivative, taken from a difference of half the step
        (yh2, _), (yl2, _) = (orc.norm(f64(x) + s * h / 2 * v64, kind, w64, None, EPS) for s in (1, -1))
        half = ((yh2 - yl2) * dy64).sum() / h
        (_, _, _), (e_dx, _, _) = orc.norm_bwd(f64(x), dy64, 0 * dy64, kind, w64, EPS)
        curve = 2 * abs(exact - half)
        assert abs(tell - slope) <= fwd_err + curve + (e_dx * np.abs(v64)).sum() + orc.STEP["fp32"] * (np.abs(f64(dx) * v64)).sum()
        (y, e) = orc.norm(f64(x), kind, np.ones(n), None, EPS)
        assert abs((f64(dw) * w64).sum() - (dy64 * y * w64).sum()) <= ((np.abs(dy64 * w64) * e).sum()
                                                                      + 20 * orc.U * np.abs(dy64 * y * w64).sum())


@pytest.mark.parametrize("n", [64, 4096])
def test_norm_strides_in_place_and_other_rows_untouched(n):
    rng = np.random.default_rng(9)
    wide, wide64 = draw(rng, 6, 3, n + 16, dtype=BF)
    w, w64 = draw(rng, n)
    x = wide[..., :n]
    want = orc.norm(wide64[..., :n].reshape(18, n), orc.LAYER, w64, None, EPS)
    out = torch.full((18, n + 8), 7.0, dtype=BF, device="cuda")
    y = rows.csa_norm(x.reshape(18, n) if not x.is_contiguous() else x, orc.LAYER, w, None, EPS)
    close(y, *want)
    rows.csa_norm(wide.view(18, n + 16)[:, :n], orc.LAYER, w, None, EPS, out=out[:, :n])
    assert torch.equal(out[:, :n], y) and bool((out[:, n:] == 7).all())
    # three dimensions that one stride reaches; in place, the gap left as it was
    gap = wide[..., n:].clone()
    assert rows.csa_norm(x, orc.LAYER, w, None, EPS, out=x) is x
    assert torch.equal(x.reshape(18, n), y) and torch.equal(wide[..., n:], gap)
    with pytest.raises(ValueError, match="row stride"):
        rows.csa_norm(wide[:, :2, :n], orc.LAYER, w, None, EPS)
    # the gradient into dout's and into x's place, one row broadcast to all
    dy, dy64 = draw(rng, 18, n, dtype=BF)
    one = y[:1].expand(18, n)
    ref = rows.csa_norm_bwd(one.contiguous(), dy, orc.RMS, w, EPS)
    got = rows.csa_norm_bwd(one, dy, orc.RMS, w, EPS)
    assert all(torch.equal(p, q) for p, q in zip(got[:2], ref[:2]))
    a, c = y.clone(), dy.clone()
    ref = rows.csa_norm_bwd(a, c, orc.LAYER, w, EPS)
    into = rows.csa_norm_bwd(a, c, orc.LAYER, w, EPS, dx=c)
    assert into[0] is c and torch.equal(c, ref[0]) and torch.equal(into[1], ref[1])
    into = rows.csa_norm_bwd(a, dy, orc.LAYER, w, EPS, dx=a)
    assert into[0] is a and torch.equal(a, ref[0]) and torch.equal(into[1], ref[1])


def test_norm_of_far_means_and_extreme_rows():
    """Means far above the spread; rows of equal channels; tiny and large magnitudes; NaN in one row only."""
    rng = np.random.default_rng(11)
    for n in (128, 4096):
        x64 = rng.standard_normal((6, n)) + 1000.0
        x64[1] *= 1e-12
        x64[2] *= 1e12
        x64[3] = 3.0
        x = torch.tensor(x64, dtype=F32, device="cuda")
        x64 = f64(x)
        for kind in (orc.RMS, orc.LAYER):
            y = rows.csa_norm(x, kind, None, None, EPS)
            close(y, *orc.norm(x64, kind, None, None, EPS), what=(n, kind))
            bad = x.clone()
            bad[5, 3] = float("nan")
            z = rows.csa_norm(bad, kind, None, None, EPS)
            assert torch.equal(z[:5], y[:5]) and bool(z[5].isnan().all())
            dz = rows.csa_norm_bwd(bad, torch.ones_like(x), kind, None, EPS)[0]
            assert torch.equal(dz[:5], rows.csa_norm_bwd(x, torch.ones_like(x), kind, None, EPS)[0][:5])


@pytest.mark.parametrize("n", [64, 2056])
@pytest.mark.parametrize("size", [1e-15, 1e-6, 1.0, 1e12])
def test_rows_of_any_size_without_eps(n, size):
    """eps = 0: the deviation is all that divides, and its cube would leave fp32."""
    rng = np.random.default_rng(37)
    x = torch.tensor((rng.standard_normal((5, n)) + 0.25) * size, dtype=F32, device="cuda")
    dy, dy64 = draw(rng, 5, n)
    w, w64 = draw(rng, n)
    rope = plan(orc.freqs(16), 0, True)
    for kind in (orc.RMS, orc.LAYER):
        close(rows.csa_norm(x, kind, w, None, 0.0), *orc.norm(f64(x), kind, w64, None, 0.0))
        want, err = orc.norm_bwd(f64(x), dy64, 0 * dy64, kind, w64, 0.0)
        for has_bias in (False, True):
            got = rows.csa_norm_bwd(x, dy, kind, w, 0.0, has_bias=has_bias)
            close(got[0], want[0], err[0], what=kind)
            close(got[1], want[1], err[1], what=kind)
        if n == 64:
            got = rows.csa_norm_rope_bwd(x[None], dy[None], kind, rope, torch.zeros(5, dtype=I32, device="cuda"), w, 0.0)
            close(got[0][0], want[0], err[0] + 6 * orc.U * (np.abs(want[0]) + np.abs(dy64 * w64).max() / size), what=kind)


@pytest.mark.parametrize("n", [128, 1024])
def test_many_rows_sum_in_a_fixed_order(n):
    """Rows for every CTA several times over: the sums against fp64, and equal bits from equal calls."""
    rng = np.random.default_rng(13)
    r = 40000 if n == 128 else 5003
    x, x64 = draw(rng, r, n, dtype=BF, shift=0.3)
    dy, dy64 = draw(rng, r, n, dtype=BF, shift=0.1)
    w, w64 = draw(rng, n)
    got = rows.csa_norm_bwd(x, dy, orc.LAYER, w, EPS, has_bias=True)
    want, err = orc.norm_bwd(x64, dy64, 0 * dy64, orc.LAYER, w64, EPS)
    for k in range(3):
        close(got[k], want[k], err[k], what=k)
    # rows of a CTA, warps and CTAs are what is summed one after another, not all rows: far below the bound
    for k in (1, 2):
        assert np.abs(f64(got[k]) - want[k]).max() <= 1e-5 * np.abs(want[k]).max()
    for _ in range(3):
        again = rows.csa_norm_bwd(x, dy, orc.LAYER, w, EPS, has_bias=True)
        assert all(torch.equal(p, q) for p, q in zip(again, got))
    only = torch.empty(n, device="cuda")
    rows.csa_norm_bwd(x, dy, orc.LAYER, None, EPS, dbias=only)
    assert torch.equal(only, got[2])


def test_sizes_beyond_32_bits_are_refused():
    """2^32 more than a size that a call takes: nothing of it may count as the small size."""
    far = 2 ** 32
    one = torch.ones(1, 1, 1, 64, device="cuda")
    before = one.clone()
    rope = plan(orc.freqs(64), 0, False)
    for axis in range(3):
        shape = [1, 1, 1, 64]
        shape[axis] += far
        x = one.expand(shape)
        for call in (lambda: rows.csa_rope(x, rope, out=x), lambda: rows.csa_rope_bwd(x, rope, dx=x),
                     lambda: rows.csa_norm_rope(x, orc.RMS, rope, out=x), lambda: rows.csa_norm_rope_bwd(x, x, orc.RMS, rope, dx=x)):
            with pytest.raises(ValueError, match="2\\^31"):
                call()
    wide = one.view(1, 64).as_strided((1, 64 + far), (1, 0))
    for call in (lambda: rows.csa_norm(wide, orc.RMS, out=wide), lambda: rows.csa_norm_bwd(wide, wide, orc.RMS, dx=wide),
                 lambda: rows.csa_norm_bwd_workspace_size(1, 64 + far)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    kv, ring, n = torch.ones(1, 1, 64, device="cuda"), torch.ones(1, 8, 64, device="cuda"), torch.ones(1, dtype=I32, device="cuda")
    for bad in (dict(ratio=4 + far), dict(coff=1 + far)):
        with pytest.raises(ValueError, match="2\\^31"):
            rows.csa_compress_decode(kv, kv, ring, ring.clone(), n, **{**dict(ratio=4), **bad})
    assert torch.equal(one, before)


# ---------------------------------------------------------------- rotation

# d, dim, first, half
TURNS = [(8, 8, 0, False), (8, 8, 0, True), (16, 4, 6, False), (64, 64, 0, True), (64, 24, 0, True), (80, 80, 0, True),
         (80, 22, 58, False), (96, 24, 72, True), (128, 128, 0, False), (128, 64, 64, True), (136, 32, 8, True), (192, 40, 2, True),
         (256, 20, 6, True), (504, 504, 0, True), (512, 512, 0, True), (512, 64, 448, False), (512, 510, 2, False), (512, 4, 508, True)]


def positions(rng, b, s, how):
    if how == "index":
        return None, np.broadcast_to(np.arange(s), (b, s))
    if how == "shared":
        p = rng.integers(-50, 5000, s)
        return torch.tensor(p, dtype=I32, device="cuda"), np.broadcast_to(p, (b, s))
    p = rng.integers(0, 1 << 20, (b, s))
    p[0, 0], p[-1, -1] = (1 << 31) - 1, -(1 << 31)
    return torch.tensor(p, dtype=I32, device="cuda"), p


@pytest.mark.parametrize("d,dim,first,half", TURNS)
def test_rope_and_norm_rope(d, dim, first, half):
    rng = np.random.default_rng(d + dim + first)
    for (b, s, H), dtype, how, scale, scaling in (((1, 1, 1), BF, "far", 1.0, "plain"), ((2, 9, 3), F32, "far", 1.25, "by_parts"),
                                                  ((3, 5, 8), BF, "shared", 0.5, "linear"), ((1, 37, 1), F32, "index", 1.0, "plain")):
        args = (dim, 10000.0, scaling, 8.0, 1024.0)
        f = orc.freqs(*args)
        rope = plan(rows.csa_rope_freqs(*args), first, half, scale)
        x, x64 = draw(rng, b, s, H, d, dtype=dtype)
        pos, p64 = positions(rng, b, s, how)
        p64 = np.broadcast_to(p64[..., None], (b, s, H))
        for inverse in (False, True):
            y = rows.csa_rope(x, rope, pos, inverse=inverse)
            close(y, *orc.turn(x64, p64, f, first, half, scale, back=inverse), what=("rope", inverse, how))
            rest = [c for c in range(d) if not first <= c < first + dim]
            assert torch.equal(y[..., rest], x[..., rest])
            z = x.clone()
            assert rows.csa_rope(z, rope, pos, inverse=inverse, out=z) is z and torch.equal(z, y)
            for dx_dt in (BF, F32):
                dx = rows.csa_rope_bwd(x, rope, pos, inverse=inverse, dx=torch.empty(x.shape, dtype=dx_dt, device="cuda"))
                close(dx, *orc.turn(x64, p64, f, first, half, scale, back=not inverse), what=("rope_bwd", inverse, how))
        w, w64 = draw(rng, d)
        c, c64 = draw(rng, d)
        for kind, bias in ((orc.RMS, None), (orc.LAYER, c)):
            n64, e = orc.norm(x64, kind, w64, None if bias is None else c64, EPS)
            t64, et = orc.turn(n64, p64, f, first, half, scale)
            y = rows.csa_norm_rope(x, kind, rope, pos, w, bias, EPS)
            close(y, t64, orc.spread(e, f, first, half, scale) + et, what=("norm_rope", kind, how))
            z = x.clone()
            assert torch.equal(rows.csa_norm_rope(z, kind, rope, pos, w, bias, EPS, out=z), y)
            for g_dt, dx_dt in ((F32, BF), (BF, F32), (BF, BF), (F32, F32)):
                dy, dy64 = draw(rng, b, s, H, d, dtype=g_dt)
                back, eb = orc.turn(dy64, p64, f, first, half, scale, back=True)
                want, err = orc.norm_bwd(x64.reshape(-1, d), back.reshape(-1, d), eb.reshape(-1, d), kind, w64, EPS)
                dx = torch.empty(x.shape, dtype=dx_dt, device="cuda")
                got = rows.csa_norm_rope_bwd(x, dy, kind, rope, pos, w, EPS, has_bias=bias is not None, dx=dx)
                close(got[0].view(-1, d), want[0], err[0], what=("norm_rope_bwd", kind, how, g_dt, dx_dt))
                close(got[1], want[1], err[1], what=("dweight", kind, how))
                assert (got[2] is None) == (bias is None)
                if bias is not None:
                    close(got[2], want[2], err[2], what=("dbias", how))


def test_rope_inverse_takes_the_rotation_back():
    """A rotation and its inverse, fp32: each is off by its bound only."""
    rng = np.random.default_rng(17)
    x, x64 = draw(rng, 2, 30, 4, 128)
    f = orc.freqs(64)
    rope = plan(f, 32, True)
    pos, p64 = positions(rng, 2, 30, "far")
    z = rows.csa_rope(rows.csa_rope(x, rope, pos), rope, pos, inverse=True)
    p64 = np.broadcast_to(p64[..., None], (2, 30, 4))
    y64, e = orc.turn(x64, p64, f, 32, True, 1.0)
    e = e + orc.STEP["fp32"] * np.abs(y64)
    _, e2 = orc.turn(y64, p64, f, 32, True, 1.0, back=True)
    close(z, x64, orc.spread(e, f, 32, True, 1.0) + e2)


def test_rows_in_other_layouts():
    """A slice of a fused projection, [H, s, b, d] memory, broadcast heads, a strided output, [b, s, d]."""
    rng = np.random.default_rng(19)
    b, s, H, d = 3, 11, 6, 128
    rope = plan(orc.freqs(64), 64, False)
    pos, _ = positions(rng, b, s, "far")
    w, _ = draw(rng, d)
    fused, _ = draw(rng, b, s, (H + 2) * d, dtype=BF)
    x = fused[..., d:(H + 1) * d].unflatten(-1, (H, d))
    ref = rows.csa_norm_rope(x.contiguous(), orc.RMS, rope, pos, w)
    assert torch.equal(rows.csa_norm_rope(x, orc.RMS, rope, pos, w), ref)
    assert torch.equal(rows.csa_rope(x, rope, pos), rows.csa_rope(x.contiguous(), rope, pos))
    big = torch.full((H, s, b, d + 8), 5.0, dtype=BF, device="cuda")
    out = big[..., :d].permute(2, 1, 0, 3)
    assert rows.csa_norm_rope(x, orc.RMS, rope, pos, w, out=out) is out
    assert torch.equal(out, ref) and bool((big[..., d:] == 5).all())
    one = x[:, :, :1].expand(b, s, H, d)
    assert torch.equal(rows.csa_norm_rope(one, orc.RMS, rope, pos, w), rows.csa_norm_rope(one.contiguous(), orc.RMS, rope, pos, w))
    dy, _ = draw(rng, H, b, s, d)
    dy = dy.permute(1, 2, 0, 3)
    got = rows.csa_norm_rope_bwd(x, dy, orc.RMS, rope, pos, w, dx=out)
    want = rows.csa_norm_rope_bwd(x.contiguous(), dy.contiguous(), orc.RMS, rope, pos, w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(rows.csa_rope_bwd(dy, rope, pos), rows.csa_rope_bwd(dy.contiguous(), rope, pos))
    k = x[:, :, 2]
    assert torch.equal(rows.csa_norm_rope(k, orc.RMS, rope, pos, w), ref[:, :, 2])
    # positions shared by the sequences, and a slice of a larger table of them
    table = torch.arange(1000, 1000 + 2 * s * b, dtype=I32, device="cuda").view(b, 2 * s)
    assert torch.equal(rows.csa_rope(x, rope, table[:, :s]), rows.csa_rope(x, rope, table[:, :s].contiguous()))
    assert torch.equal(rows.csa_rope(x, rope, table[1, :s]), rows.csa_rope(x, rope, table[1:2, :s].expand(b, s).contiguous()))
    assert torch.equal(rows.csa_rope(x, rope, table[:1, :s].expand(b, s)), rows.csa_rope(x, rope, table[0, :s]))


def test_infinities_stay_in_their_pairs():
    """Channels that are not turned keep their bits; a pair's NaN reaches no other pair."""
    x = torch.zeros(1, 2, 1, 128, dtype=BF, device="cuda")
    x[0, 0, 0, [0, 7, 66, 127]] = torch.tensor([float("inf"), float("nan"), float("-inf"), 1.0], dtype=BF, device="cuda")
    rope = plan(orc.freqs(22), 64, False)         # channels 64 .. 85
    y = rows.csa_rope(x, rope)
    assert y[0, 0, 0, 0].item() == float("inf") and bool(y[0, 0, 0, 7].isnan()) and y[0, 0, 0, 127].item() == 1
    finite = [c for c in range(128) if c not in (0, 7, 66, 67)]
    assert bool(y[0, 0, 0, finite].isfinite().all()) and bool((y[0, 1] == 0).all())


def test_empty_calls():
    rope = plan(orc.freqs(8), 0, False)
    for shape in ((0, 4, 2, 8), (2, 0, 2, 8), (2, 4, 0, 8)):
        x = torch.empty(shape, dtype=BF, device="cuda")
        assert rows.csa_rope(x, rope).shape == shape == rows.csa_norm_rope(x, orc.RMS, rope).shape
        w = torch.ones(8, device="cuda")
        dx, dw, db = rows.csa_norm_rope_bwd(x, x, orc.RMS, rope, None, w, has_bias=True)
        assert dx.shape == shape and dw.tolist() == [0.0] * 8 == db.tolist()
    x = torch.empty(0, 4096, device="cuda")
    w = torch.ones(4096, device="cuda")
    dx, dw, db = rows.csa_norm_bwd(x, x, orc.LAYER, w, has_bias=True)
    assert rows.csa_norm(x, orc.RMS).shape == x.shape == dx.shape and not dw.any() and not db.any()


# ----------------------------------------------------- streams and graphs

def test_other_streams_and_replayed_graphs():
    rng = np.random.default_rng(23)
    rope = plan(orc.freqs(128), 0, True)
    w, _ = draw(rng, 128)
    wide, _ = draw(rng, 4096)
    pos = torch.zeros(2, 40, dtype=I32, device="cuda")

    def step(x, h):
        y = rows.csa_norm_rope(x, orc.RMS, rope, pos, w)
        return (y, rows.csa_rope(y, rope, pos, inverse=True), *rows.csa_norm_rope_bwd(x, y, orc.LAYER, rope, pos, w, has_bias=True),
                rows.csa_norm(h, orc.LAYER, wide), *rows.csa_norm_bwd(h, h, orc.RMS, wide)[:2])

    inputs = [(draw(rng, 2, 40, 8, 128, dtype=BF)[0], draw(rng, 300, 4096, dtype=BF)[0]) for _ in range(3)]
    want = [[t.clone() for t in step(*i)] for i in inputs]
    x, h = (t.clone() for t in inputs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rows.csa_norm_rope_bwd(x, x, orc.LAYER, rope, pos, w, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got[:2], rows.csa_norm_rope_bwd(x, x, orc.LAYER, rope, pos, w)[:2]))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step(x, h)
        graphs.append((g, res))
    for i, (xi, hi) in enumerate(inputs + inputs[:1]):
        x.copy_(xi)
        h.copy_(hi)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, res in graphs:
            assert all(torch.equal(p, q) for p, q in zip(res, want[i % 3]))


FIRST_CALLS = """
import sys
sys.path[:0] = {path!r}
import torch
from compressed_sparse_attention_sum_gb300 import csa, rows
g = torch.Generator(device="cuda").manual_seed(0)
f = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
half = rows.CsaRope(rows.csa_rope_turns(rows.csa_rope_freqs(128)), 0, "half")
inter = rows.CsaRope(rows.csa_rope_turns(rows.csa_rope_freqs(64)), 64)
x, h, wide, w = f(2, 30, 8, 128).bfloat16(), f(300, 4096).bfloat16(), f(4096), f(128)
kv, score, rings = f(2, 9, 128).bfloat16(), f(2, 9, 128).bfloat16(), [torch.zeros(2, 16, 128, device="cuda").bfloat16() for _ in range(2)]
lens = torch.full((2,), 9, dtype=torch.int32, device="cuda")
out = torch.zeros(2, 3, 128, device="cuda").bfloat16()
def step():
    y = rows.csa_norm_rope(x, 1, half, None, w)
    r = rows.csa_compress_decode(kv, score, *rings, lens, 4, 2, 1, w, None, 1e-6, inter, out=out)
    return [y, rows.csa_rope(y, inter), rows.csa_rope_bwd(y, inter), *rows.csa_norm_rope_bwd(x, y, 2, half, None, w, has_bias=True),
            rows.csa_norm(h, 2, wide), *rows.csa_norm_bwd(h, h, 1, wide)[:2], *(t.clone() for t in r)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert csa.csa_get_device_status() == 0
assert all(torch.equal(x, y) for x, y in zip(got, step()))
print("same")
"""


def test_the_first_calls_of_a_process_can_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(path=sys.path)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]


def test_offsets_beyond_32_bits():
    """Rows 2^31 elements and more apart, in and out."""
    rng = np.random.default_rng(29)
    far = (1 << 31) + 64
    big = torch.empty(3 * far, dtype=BF, device="cuda")
    rope, w = plan(orc.freqs(64), 64, True), draw(rng, 4096)[0]
    for n in (128, 4096):
        src, _ = draw(rng, 2, n, dtype=BF)
        x, y = big.as_strided((2, n), (far, 1)), big.as_strided((2, n), (far, 1), 8192)
        x.copy_(src)
        rows.csa_norm(x, orc.LAYER, w[:n], None, EPS, out=y)
        assert torch.equal(y, rows.csa_norm(src, orc.LAYER, w[:n], None, EPS))
        got = rows.csa_norm_bwd(x, x, orc.LAYER, w[:n], EPS, has_bias=True, dx=y)
        assert all(torch.equal(p, q) for p, q in zip(got, rows.csa_norm_bwd(src, src, orc.LAYER, w[:n], EPS, has_bias=True)))
    src, _ = draw(rng, 2, 3, 5, 128, dtype=BF)
    pos = torch.tensor([7, 1 << 30, 9], dtype=I32, device="cuda")
    for strides in ((far, 640, 128), (128, far // 2, 256), (640, 128 * 16, far // 4)):
        x, y = big.as_strided((2, 3, 5, 128), (*strides, 1)), big.as_strided((2, 3, 5, 128), (*strides, 1), 8192 * 4)
        x.copy_(src)
        rows.csa_norm_rope(x, orc.RMS, rope, pos, w[:128], out=y)
        want = rows.csa_norm_rope(src, orc.RMS, rope, pos, w[:128])
        assert torch.equal(y, want)
        got = rows.csa_norm_rope_bwd(x, x, orc.RMS, rope, pos, w[:128], dx=y)
        assert all(torch.equal(p, q) for p, q in zip(got[:2], rows.csa_norm_rope_bwd(src, src, orc.RMS, rope, pos, w[:128])[:2]))


def test_two_streams_at_once():
    """The same calls on two streams, each with a workspace of its own."""
    rng = np.random.default_rng(31)
    rope = plan(orc.freqs(128), 0, False)
    w, _ = draw(rng, 128)
    wide, _ = draw(rng, 2056)
    sets = [(draw(rng, 4, 200, 8, 128, dtype=BF)[0], draw(rng, 700, 2056)[0]) for _ in range(2)]

    def step(x, h):
        return [*rows.csa_norm_rope_bwd(x, x, orc.LAYER, rope, None, w, has_bias=True), *rows.csa_norm_bwd(h, h, orc.LAYER, wide, has_bias=True),
                rows.csa_norm_rope(x, orc.RMS, rope, None, w), rows.csa_norm(h, orc.RMS, wide)]

    want = [[t.clone() for t in step(*s)] for s in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for res in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(res, want[i]))


def test_strides_of_an_empty_tensor_are_not_taken_for_anothers():
    rope = plan(orc.freqs(8), 0, False)
    base = torch.zeros(4, 4, 16, 8, dtype=BF, device="cuda")
    turned = base.transpose(2, 3)                  # rows of 16 channels, 8 apart
    rows.csa_rope(turned[:0], rope, out=turned[:0].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        rows.csa_rope(turned, rope)


def test_the_binding_refuses():
    x = torch.zeros(2, 3, 4, 64, dtype=BF, device="cuda")
    rope = plan(orc.freqs(64), 0, False)
    f = torch.ones(64, device="cuda")
    bad = [lambda: rows.csa_norm(x.half(), orc.RMS), lambda: rows.csa_norm(x, orc.RMS, f.bfloat16()), lambda: rows.csa_norm(x, orc.RMS, f[:32]),
           lambda: rows.csa_norm(x, orc.RMS, f.cpu()), lambda: rows.csa_norm(x, orc.RMS, out=x.float()), lambda: rows.csa_norm(x.transpose(2, 3), orc.RMS),
           lambda: rows.csa_norm(x, 0), lambda: rows.csa_norm(x, orc.RMS, eps=-1.0), lambda: rows.csa_norm_bwd(x, x[:1], orc.RMS),
           lambda: rows.csa_norm_bwd(x, x, orc.RMS, f, workspace=torch.empty(0, dtype=torch.uint8, device="cuda")),
           lambda: rows.csa_rope(x, None), lambda: rows.csa_rope(x, rope, torch.zeros(2, 3, device="cuda")),
           lambda: rows.csa_rope(x, rope, torch.zeros(3, 2, dtype=I32, device="cuda")), lambda: rows.csa_rope(x, plan(orc.freqs(62), 4, False)),
           lambda: rows.csa_rope(x, plan(orc.freqs(8), 1, False)), lambda: rows.csa_rope(x, plan(orc.freqs(6), 0, True)),
           lambda: rows.csa_rope(x, rope, out=torch.zeros_like(x[:, :, :1]).expand_as(x)), lambda: rows.csa_rope(x[0, 0], rope),
           lambda: rows.csa_norm_rope(x, orc.RMS, rope, weight=f[None]), lambda: rows.csa_rope_bwd(x, rope, dx=x.cpu()),
           lambda: plan(orc.freqs(8), 0, False, float("nan")) and rows.csa_rope(x, plan(orc.freqs(8), 0, False, float("nan")))]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, csa.CSAError)):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(AttributeError):
        rope.first = 8


def test_channels_that_are_not_turned_keep_their_values():
    """Any bits: infinities, zeros of both signs and subnormal values stay as they are, NaNs stay NaNs; out of place, in place and
    turned back, in vectors that turn in part, in whole or not at all."""
    rng = np.random.default_rng(41)
    for dtype, bits in ((BF, torch.int16), (F32, torch.int32)):
        top = 1 << 8 * dtype.itemsize
        for d, dim, first, half in TURNS:
            rest = [c for c in range(d) if not first <= c < first + dim]
            rope = plan(orc.freqs(dim), first, half)
            for b, s, H in ((1, 3, 1), (2, 5, 6)):
                odd = torch.tensor(rng.integers(-top // 2, top // 2, (b, s, H, d)), dtype=bits, device="cuda")
                odd[0, 0, 0, :4] = torch.tensor([float("inf"), float("-inf"), 0.0, -0.0], dtype=dtype).view(bits).cuda()
                odd[..., first:first + dim] = draw(rng, b, s, H, dim, dtype=dtype)[0].view(bits)
                x = odd.view(dtype)
                nan = x[..., rest].isnan()
                for inverse in (False, True):
                    outs = [rows.csa_rope(x, rope, inverse=inverse), rows.csa_rope_bwd(x, rope, inverse=inverse)]
                    z = x.clone()
                    outs.append(rows.csa_rope(z, rope, inverse=inverse, out=z))
                    for y in outs:
                        at = (dtype, d, dim, first, half, inverse)
                        assert torch.equal(y[..., rest].isnan(), nan), at
                        assert torch.equal(y.view(bits)[..., rest][~nan], odd[..., rest][~nan]), at
                        assert bool(y[..., first:first + dim].isfinite().all()), at


def test_numbers_beyond_32_bits_are_not_cut():
    """A kind and a first channel that are a good one and 2^32."""
    x, ring, lens = torch.ones(1, 8, 64, device="cuda"), torch.ones(1, 8, 64, device="cuda"), torch.ones(1, dtype=I32, device="cuda")
    turns, far = rows.csa_rope_turns(orc.freqs(64)), 2 ** 32
    rope = rows.CsaRope(turns)
    for first in (far, -far, -2):
        with pytest.raises(ValueError, match="first"):
            rows.CsaRope(turns, first)
    for kind in (1 + far, 2 - far):
        for call in (lambda: rows.csa_norm(x, kind), lambda: rows.csa_norm_bwd(x, x, kind), lambda: rows.csa_norm_rope(x, kind, rope),
                     lambda: rows.csa_norm_rope_bwd(x, x, kind, rope),
                     lambda: rows.csa_compress_decode(x, x, ring, ring.clone(), lens, 4, kind=kind)):
            with pytest.raises(ValueError, match="kind"):
                call()
