"""The whole-sequence compressors and their gradients with scores that mask tokens or have a
common offset, against the fp64 oracle (bounds as oracle/rows_oracle.py derives them)."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_sum_gb300 import csa
from oracle import csa_oracle as whole
from oracle import rows_oracle as orc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAME = {BF: "bf16", F32: "fp32"}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from compressed_sparse_attention_sum_gb300 import build
    build.build()
    csa.load_library()
    csa.csa_get_device_status()
    yield
    assert csa.csa_get_device_status() == 0


def f64(t):
    return t.detach().double().cpu().numpy()


def gradient_bounds(kv, score, ratio, coff, g):
    """Bounds of the fp32 errors of (dkv, dscore) of one sequence kv [n, d], score [n, d or 1], g [n / ratio, d]: a weight is off as
    orc.compress counts it, the products and sums by their own roundings, a shared score's sum over channels by D."""
    e_kv, e_s, size = np.zeros_like(kv), np.zeros_like(kv), np.zeros_like(kv)
    for j in range(kv.shape[0] // ratio):
        t = whole.pooling_window(j, ratio, coff)
        z = np.broadcast_to(score[t], kv[t].shape)
        w = np.exp(z - z.max(0))
        w = w / w.sum(0)
        far = np.where(w > 0, w * np.where(w > 0, z.max(0) - z, 0.0), 0.0)
        e_w = orc.U * (3 * far + w * (3 * far.sum(0) + 24 + 2 * orc.D))
        pooled, e_p = (w * kv[t]).sum(0), (e_w * np.abs(kv[t])).sum(0) + 2 * orc.D * orc.U * (w * np.abs(kv[t])).sum(0)
        e_kv[t] += np.abs(g[j]) * (e_w + 4 * orc.U * w)
        apart = np.abs(kv[t] - pooled)
        e_s[t] += np.abs(g[j]) * (e_w * apart + w * e_p + 6 * orc.U * w * (np.abs(kv[t]) + np.abs(pooled)))
        size[t] += np.abs(g[j]) * w * apart
    if score.shape[1] == 1:
        e_s = (e_s + orc.D * orc.U * size).sum(1, keepdims=True)
    return e_kv, e_s


def check(ratio, coff, dtype, sw, d, n, change):
    """csa_compress_overlap and its gradient with scores that `change` alters, for two sequences."""
    g = torch.Generator().manual_seed(ratio + d)
    kv = torch.randn(2, n, d, generator=g).to(dtype).cuda()
    score = (1.5 * torch.randn(2, n, d if sw == "d" else 1, generator=g)).to(dtype).cuda()
    dout = torch.randn(2, n // ratio, d, generator=g).cuda()
    change(score)
    out = csa.csa_compress_overlap(kv, score, ratio, coff)
    dkv = torch.ones(2, n, d, device="cuda")
    dscore = csa.csa_compress_overlap_bwd(kv, score, ratio, coff, dout, dkv)
    want_kv, want_s = whole.compress_bwd(f64(kv), f64(score), ratio, f64(dout), coff)
    for i in range(2):
        want, err = orc.compress(f64(kv[i]), f64(score[i]), ratio, coff, 0, None, None, 0.0, None, 0, False, 1.0, NAME[dtype])
        e_kv, e_s = gradient_bounds(f64(kv[i]), f64(score[i]), ratio, coff, f64(dout[i]))
        for what, got, ref, e in (("out", out[i], want, err + orc.STEP[NAME[dtype]] * (np.abs(want) + err)),
                                  ("dkv", dkv[i], 1 + want_kv[i], e_kv + orc.U * (1 + np.abs(want_kv[i])) * (coff + 1)),
                                  ("dscore", dscore[i], want_s[i], e_s + orc.U * np.abs(want_s[i]))):
            off = np.abs(f64(got) - ref) / (e + 1e-30)
            assert np.isfinite(f64(got)).all() and off.max() <= 1, (what, i, float(off.max()))


SHAPES = [(4, 1, 64), (7, 1, 64), (16, 1, 512), (128, 1, 128), (300, 1, 72), (4, 2, 128), (20, 2, 64)]
LOWEST = "lowest of the type"


@pytest.mark.parametrize("value", [-1e4, -1e10, -1e30, LOWEST])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ratio,coff,d", SHAPES)
def test_scores_masked_by_a_finite_value(ratio, coff, d, dtype, value):
    """Whole blocks (their mean is what the softmax gives), the start of one, tokens in the middle, all but one."""
    n = 5 * ratio + 1
    mask = torch.zeros(n, dtype=torch.bool)
    mask[:ratio + (ratio + 1) // 2] = True
    mask[2 * ratio + 1:3 * ratio] = True
    mask[3 * ratio:4 * ratio:2] = True

    def change(score):
        score[1, mask.cuda()] = torch.finfo(dtype).min if value is LOWEST else value

    for sw in ("d", 1):
        check(ratio, coff, dtype, sw, d, n, change)


@pytest.mark.parametrize("offset", [300.0, -30000.0, 1e9, -1e30])
@pytest.mark.parametrize("ratio,coff,d", SHAPES)
def test_a_common_offset_of_the_scores(ratio, coff, d, offset):
    check(ratio, coff, F32, "d", d, 3 * ratio, lambda score: score.add_(offset))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ratio,coff,d", SHAPES)
def test_scores_of_minus_infinity(ratio, coff, d, dtype):
    """The start of a block, tokens in the middle, all but one."""
    n = 4 * ratio
    mask = torch.zeros(n, dtype=torch.bool)
    for j in range(4):
        at = slice(j * ratio, (j + 1) * ratio)
        mask[at] = torch.tensor([(t < ratio // 2, t % 2 == 0, t != ratio - 1, t != 0)[j] for t in range(ratio)])
    for sw in ("d", 1):
        check(ratio, coff, dtype, sw, d, n, lambda score: score[1].masked_fill_(mask.cuda()[:, None], float("-inf")))


@pytest.mark.parametrize("ratio,coff,d", SHAPES)
def test_a_window_of_minus_infinities(ratio, coff, d):
    """A channel whose scores are all -inf has no weights: NaN there, and nowhere else."""
    n = (coff + 2) * ratio
    g = torch.Generator().manual_seed(3)
    kv, score = torch.randn(1, n, d, generator=g).cuda(), torch.randn(1, n, d, generator=g).cuda()
    want = csa.csa_compress_overlap(kv, score, ratio, coff)
    score[:, :coff * ratio, 5] = float("-inf")
    got = csa.csa_compress_overlap(kv, score, ratio, coff)
    none = torch.zeros_like(got, dtype=torch.bool)
    none[:, :coff, 5] = True
    assert torch.equal(got.isnan(), none)
    none[:, :, 5] = True
    assert torch.equal(got[~none], want[~none])
    w = torch.ones(d, device="cuda")
    rows = csa.csa_compress_norm_rope(kv, score, ratio, w, 1e-6, 0, 1e4)
    assert bool(rows[:, :coff].isnan().all()) and bool(rows[:, coff:].isfinite().all())
