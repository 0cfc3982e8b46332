"""The row calls on more rows than the GPU holds at once, where a lane or a CTA goes through
many rows and each place of shared memory is used again: every row has the bits that a call on
few rows gives it (those calls are compared with the fp64 oracle in test_gpu_row_calls.py), rows
from all over against the oracle, and the sums over rows against fp64."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_sum_gb300 import csa, rows
from oracle import rows_oracle as orc
from test_gpu_row_calls import BF, EPS, F32, I32, close, draw, f64, plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from compressed_sparse_attention_sum_gb300 import build
    build.build()
    rows.load_library()
    csa.csa_get_device_status()
    yield
    assert csa.csa_get_device_status() == 0


def many(seed, *shape, dtype=BF, shift=0.0):
    """Rows made on the GPU, with channels of different size and mean."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda")) + shift
    return x.to(dtype)


def some(n, seed):
    """Numbers below n: the first, the last and others."""
    return np.unique(np.concatenate(([0, n - 1], np.random.default_rng(seed).integers(0, n, 300))))


def spun(x, pos, f, first, half):
    """Rows [rows, d] turned back by positions [rows], and a bound of the fp32 error (as orc.turn), in fp64 on the GPU."""
    u, v = (torch.tensor(i, device="cuda") for i in orc.pairs(2 * len(f), first, half))
    angle = pos.double()[:, None] * torch.tensor(f, device="cuda")
    c, s, x = angle.cos(), angle.sin(), x.double()
    y, err = x.clone(), torch.zeros_like(x)
    y[:, u], y[:, v] = x[:, u] * c + x[:, v] * s, x[:, v] * c - x[:, u] * s
    err[:, u] = err[:, v] = (x[:, u].abs() + x[:, v].abs()) * (6 * orc.U + angle.abs() * 2.0 ** -51)
    return y, err


def sums(x, dy, kind, chain, turned=None):
    """((dweight, bound), (dbias, bound)) of rows [rows, n] in fp64: `chain` additions one after another, and the errors of a row's
    own terms as orc.norm_bwd counts them.  turned: dy's rows i .. j - 1 turned back, with their errors."""
    dw, db, size_w, size_b, off_w, off_b = (torch.zeros(x.shape[1], dtype=torch.float64, device="cuda") for _ in range(6))
    for i in range(0, x.shape[0], 16384):
        a, g = x[i:i + 16384].double(), dy[i:i + 16384].double()
        eg = torch.zeros_like(g)
        if turned is not None:
            g, eg = turned(i, i + 16384)
        m = a.mean(-1, keepdim=True) if kind == orc.LAYER else 0 * a[:, :1]
        r = 1 / torch.sqrt(((a - m) ** 2).mean(-1, keepdim=True) + EPS)
        xh = (a - m) * r
        e_m = orc.D * orc.U * a.abs().mean(-1, keepdim=True) * (kind == orc.LAYER)
        ex = e_m * r + xh.abs() * ((orc.D / 2 + 10) * orc.U + 0.5 * (e_m * r) ** 2)
        dw, db = dw + (g * xh).sum(0), db + g.sum(0)
        size_w, size_b = size_w + (g * xh).abs().sum(0), size_b + g.abs().sum(0)
        off_w, off_b = off_w + (g.abs() * ex + eg * xh.abs()).sum(0), off_b + eg.sum(0)
    return (f64(dw), f64(off_w + chain * orc.U * size_w)), (f64(db), f64(off_b + chain * orc.U * size_b))


# rows of at most 4096 channels by the thousand have kernels of their own, which few rows do not reach: all rows
# against the oracle.  Each CTA has more rows than it holds in flight; the last ones are no whole round.
FEW_KERNELS = [(520, 8701), (1000, 6701), (1024, 305), (1024, 6701), (1032, 4501), (2048, 4501), (2056, 3001), (4096, 305), (4096, 2501)]


@pytest.mark.parametrize("kind", [orc.RMS, orc.LAYER])
@pytest.mark.parametrize("n,count", FEW_KERNELS)
def test_norm_of_many_rows(n, count, kind):
    rng = np.random.default_rng(n + count + kind)
    w, w64 = draw(rng, n)
    b, b64 = draw(rng, n)
    for dtype in (BF, F32):
        x = many(count + n, count, n, dtype=dtype, shift=0.5)
        y = rows.csa_norm(x, kind, w, b, EPS)
        close(y, *orc.norm(f64(x), kind, w64, b64, EPS), what=(n, count, kind, dtype))
        z = x.clone()
        assert rows.csa_norm(z, kind, w, b, EPS, out=z) is z and torch.equal(z, y)


@pytest.mark.parametrize("kind", [orc.RMS, orc.LAYER])
@pytest.mark.parametrize("n,count", [(8, 200001), (64, 400003), (128, 300007), (200, 100003), (512, 90001), (4104, 1601), (8192, 1601),
                                     (8200, 903), (16384, 903), (16392, 620), (32768, 620)])
def test_norm_of_many_rows_has_the_bits_of_few(n, count, kind):
    rng = np.random.default_rng(n + kind)
    w, w64 = draw(rng, n)
    b, b64 = draw(rng, n)
    step = 1021 if n <= 512 else 152
    for dtype in (BF, F32):
        x = many(count + n, count, n, dtype=dtype, shift=0.5)
        y = rows.csa_norm(x, kind, w, b, EPS)
        for i in range(0, count, step):
            assert torch.equal(y[i:i + step], rows.csa_norm(x[i:i + step], kind, w, b, EPS)), (i, dtype)
        at = some(count, n)
        close(y[at], *orc.norm(f64(x[at]), kind, w64, b64, EPS), what=(n, count, kind, dtype))


@pytest.mark.parametrize("kind", [orc.RMS, orc.LAYER])
@pytest.mark.parametrize("n,count", [(64, 100003), (512, 40001), (520, 9001), (1024, 5003), (2048, 3001), (2056, 3001), (4096, 1601), (7168, 903),
                                     (8192, 903), (16384, 620), (32768, 471)])
def test_gradient_of_many_rows(n, count, kind):
    rng = np.random.default_rng(n + kind)
    w, w64 = draw(rng, n)
    step = 1021 if n <= 512 else 152
    for dtype, g_dt in ((BF, BF), (F32, F32), (BF, F32), (F32, BF)):
        x, dy = many(n, count, n, dtype=dtype, shift=0.5), many(n + 1, count, n, dtype=g_dt)
        for has_bias in (False, True):
            dx, dw, db = rows.csa_norm_bwd(x, dy, kind, w, EPS, has_bias=has_bias)
            for i in range(0, count, step):
                few = rows.csa_norm_bwd(x[i:i + step], dy[i:i + step], kind, w, EPS, has_bias=has_bias)[0]
                assert torch.equal(dx[i:i + step], few), (i, dtype, g_dt)
            # a CTA's rows in turn (152 CTAs at least), then its warps, then at most 76 CTAs' shares in a warp, then the warps
            (want_w, e_w), (want_b, e_b) = sums(x, dy, kind, count // 152 + 1 + 8 + 76 + 8)
            close(dw, want_w, e_w, what=(n, dtype, g_dt))
            assert (db is None) == (not has_bias)
            if has_bias:
                close(db, want_b, e_b, what=(n, dtype, g_dt))
            at = some(count, n)
            want, err = orc.norm_bwd(f64(x[at]), f64(dy[at]), 0 * f64(dy[at]), kind, w64, EPS)
            close(dx[at], want[0], err[0], what=(n, dtype, g_dt))
        z = dy.clone()
        assert torch.equal(rows.csa_norm_bwd(x, z, kind, w, EPS, has_bias=True, dx=z)[0], z)
        assert torch.equal(rows.csa_norm_bwd(x, dy, kind, w, EPS, has_bias=True, dx=torch.empty_like(dy))[0], z)


# b, s, H, d, dim, first, half: runs of 16 heads and more than one round of them; few heads; the tokens of one head, or
# of two or three; pairs on vectors of 16 bytes and on smaller ones
TURNED = [(2, 4097, 32, 128, 128, 0, True), (3, 3001, 5, 512, 64, 448, False), (1, 1801, 64, 512, 64, 448, False), (1, 60013, 1, 128, 128, 0, True),
          (2, 20011, 3, 64, 22, 42, False), (2, 9001, 2, 80, 40, 0, True), (1, 3001, 8, 192, 40, 2, True), (5, 8003, 1, 512, 64, 448, False),
          (2, 1001, 20, 256, 256, 0, False), (1, 2113, 64, 512, 64, 448, False), (3, 3001, 64, 128, 64, 64, False)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", TURNED, ids=str)
def test_rotations_of_many_rows(case, dtype):
    b, s, H, d, dim, first, half = case
    rng = np.random.default_rng(s)
    f = orc.freqs(dim)
    rope = plan(f, first, half, 1.25)
    w, w64 = draw(rng, d)
    c, c64 = draw(rng, d)
    x = many(s, b, s, H, d, dtype=dtype, shift=0.3)
    pos = torch.tensor(rng.integers(-100, 1 << 20, (b, s)), dtype=I32, device="cuda")
    step = max(1, 2000 // (b * H))

    def forward(x, pos):
        return [rows.csa_rope(x, rope, pos), rows.csa_rope(x, rope, pos, inverse=True),
                rows.csa_rope_bwd(x, rope, pos, dx=torch.empty(x.shape, dtype=F32 if dtype is BF else BF, device="cuda")),
                rows.csa_norm_rope(x, orc.RMS, rope, pos, w, None, EPS), rows.csa_norm_rope(x, orc.RMS, rope, pos, w, c, EPS),
                rows.csa_norm_rope(x, orc.LAYER, rope, pos, w, c, EPS)]

    got = forward(x, pos)
    for t in range(0, s, step):
        few = forward(x[:, t:t + step], pos[:, t:t + step])
        for k in range(len(got)):
            assert torch.equal(got[k][:, t:t + step], few[k]), (k, t)
    z = x.clone()
    assert torch.equal(rows.csa_rope(z, rope, pos, out=z), got[0])
    assert torch.equal(rows.csa_norm_rope(x, orc.RMS, rope, None, w, None, EPS),
                       rows.csa_norm_rope(x, orc.RMS, rope, torch.arange(s, dtype=I32, device="cuda"), w, None, EPS))
    at = some(b * s * H, s)
    x64 = f64(x.reshape(-1, d)[at])
    p64 = f64(pos.reshape(-1))[at // H]
    for k, back in ((0, False), (1, True), (2, True)):
        close(got[k].reshape(-1, d)[at], *orc.turn(x64, p64, f, first, half, 1.25, back=back), what=(case, k))
    for k, kind, bias in ((3, orc.RMS, None), (4, orc.RMS, c64), (5, orc.LAYER, c64)):
        y64, e = orc.norm(x64, kind, w64, bias, EPS)
        t64, et = orc.turn(y64, p64, f, first, half, 1.25)
        close(got[k].reshape(-1, d)[at], t64, orc.spread(e, f, first, half, 1.25) + et, what=(case, k))


@pytest.mark.parametrize("dtype,g_dt", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("case", TURNED, ids=str)
def test_gradient_of_many_turned_rows(case, dtype, g_dt):
    b, s, H, d, dim, first, half = case
    rng = np.random.default_rng(s)
    f = orc.freqs(dim)
    rope = plan(f, first, half)
    w, w64 = draw(rng, d)
    x, dy = many(s, b, s, H, d, dtype=dtype, shift=0.3), many(s + 1, b, s, H, d, dtype=g_dt)
    pos = torch.tensor(rng.integers(-100, 1 << 20, (b, s)), dtype=I32, device="cuda")
    step = max(1, 2000 // (b * H))
    flat, at_row = dy.reshape(-1, d), pos.reshape(-1).repeat_interleave(H)
    for kind, has_bias in ((orc.RMS, False), (orc.RMS, True), (orc.LAYER, True)):
        dx, dw, db = rows.csa_norm_rope_bwd(x, dy, kind, rope, pos, w, EPS, has_bias=has_bias)
        for t in range(0, s, step):
            few = rows.csa_norm_rope_bwd(x[:, t:t + step], dy[:, t:t + step], kind, rope, pos[:, t:t + step], w, EPS, has_bias=has_bias)
            assert torch.equal(dx[:, t:t + step], few[0]), t
        # as in test_gradient_of_many_rows (a lane has an eighth of a CTA's rows at most)
        (want_w, e_w), (want_b, e_b) = sums(x.reshape(-1, d), flat, kind, b * s * H // 152 + 1 + 8 + 76 + 8,
                                            lambda i, j: spun(flat[i:j], at_row[i:j], f, first, half))
        close(dw, want_w, e_w, what=(case, kind))
        assert (db is None) == (not has_bias)
        if has_bias:
            close(db, want_b, e_b, what=(case, kind))
        at = some(b * s * H, s)
        p64 = f64(pos.reshape(-1))[at // H]
        g64, eb = orc.turn(f64(dy.reshape(-1, d)[at]), p64, f, first, half, 1.0, back=True)
        want, err = orc.norm_bwd(f64(x.reshape(-1, d)[at]), g64, eb, kind, w64, EPS)
        close(dx.reshape(-1, d)[at], want[0], err[0], what=(case, kind))
