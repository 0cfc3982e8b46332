"""csa_compress_decode on the GPU: against the fp64 oracle, against the whole-sequence
calls, token by token, in chunks and with tokens taken back, and a decode loop of a
layer whose rows are normalised and turned, captured into one graph."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_sum_gb300 import csa, rows, serve
from oracle import rows_oracle as orc

pytestmark = pytest.mark.gpu

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
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
    return t.detach().double().cpu().numpy()


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Layer:
    """A compressor with its inputs for b sequences of n tokens."""

    def __init__(self, seed, b, n, d, ratio, coff, sw, dtype, kind=orc.RMS, dim=32, half=False, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.b, self.n, self.d, self.ratio, self.coff, self.dtype, self.kind = b, n, d, ratio, coff, dtype, kind
        self.kv = torch.randn(b, n, d, generator=g).to(dtype).cuda()
        self.score = (1.5 * torch.randn(b, n, d if sw == "d" else 1, generator=g)).to(dtype).cuda()
        self.weight = (0.5 + torch.rand(d, generator=g)).cuda() if kind else None
        self.bias = torch.randn(d, generator=g).cuda() if kind == orc.LAYER else None
        self.f = orc.freqs(dim, 40000.0) if dim else None
        self.first, self.half, self.scale = d - dim, half, scale
        self.rope = rows.CsaRope(rows.csa_rope_turns(self.f), d - dim, "half" if half else "interleaved", scale) if dim else None

    def rings(self, R):
        """Rings of R rows that hold nothing yet (NaN: whatever they hold must not matter)."""
        nan = float("nan")
        return (torch.full((self.b, R, self.d), nan, dtype=self.dtype, device="cuda"),
                torch.full((self.b, R, self.score.shape[2]), nan, dtype=self.dtype, device="cuda"))

    def call(self, rings, at, s, out=None, lens=None, **kw):
        """The call for tokens at .. at + s - 1 of every sequence."""
        kv, score = self.kv[:, at:at + s], self.score[:, at:at + s]
        lens = ints([at + s] * self.b) if lens is None else lens
        return rows.csa_compress_decode(kv, score, *rings, lens, self.ratio, self.coff, self.kind, self.weight, self.bias, EPS, self.rope,
                                        out=out, **kw)

    def run(self, rings, sizes):
        """Tokens in calls of the given sizes; the rows of all blocks [b, n / ratio, d]."""
        got = torch.full((self.b, sum(sizes) // self.ratio, self.d), 9.0, dtype=self.dtype, device="cuda")
        at = 0
        for s in sizes:
            out, first, counts = self.call(rings, at, s)
            j, k = at // self.ratio, (at + s) // self.ratio - at // self.ratio
            assert first.tolist() == [j] * self.b and counts.tolist() == [k] * self.b
            got[:, j:j + k] = out[:, :k]
            at += s
        return got

    def oracle(self, i, n):
        opt = lambda t: None if t is None else f64(t)  # noqa: E731
        return orc.compress(f64(self.kv[i, :n]), f64(self.score[i, :n]), self.ratio, self.coff, self.kind, opt(self.weight), opt(self.bias),
                            EPS, self.f, self.first, self.half, self.scale, NAME[self.dtype])


def close(got, want, err, dtype):
    g = f64(got)
    off = np.abs(g - want) / (err + orc.STEP[NAME[dtype]] * (np.abs(want) + err) + 1e-37)
    assert np.isfinite(g).all() and off.max(initial=0) <= 1, float(off.max())


CASES = [
    # b, n, d, ratio, coff, score width, dtype, kind, dim, half
    (1, 9, 8, 1, 1, "d", F32, orc.RMS, 8, False),
    (2, 23, 64, 4, 1, "d", BF, orc.RMS, 32, False),
    (2, 23, 64, 4, 2, 1, F32, orc.LAYER, 64, True),
    (3, 31, 128, 4, 2, "d", BF, orc.LAYER, 24, True),
    (2, 50, 136, 7, 2, "d", F32, orc.RMS, 22, False),
    (1, 300, 128, 128, 1, "d", BF, orc.RMS, 64, False),
    (1, 300, 80, 100, 2, 1, BF, 0, 0, False),
    (2, 40, 512, 4, 2, "d", BF, orc.RMS, 64, False),
    (1, 270, 512, 128, 1, "d", F32, orc.LAYER, 512, True),
    (1, 40, 504, 16, 1, "d", F32, orc.RMS, 6, False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_blocks_against_the_oracle_however_the_tokens_come(case):
    b, n, d, ratio, coff, sw, dtype, kind, dim, half = case
    L = Layer(31, b, n, d, ratio, coff, sw, dtype, kind, dim, half, scale=1.25 if half else 1.0)
    R = coff * ratio - 1 + n
    whole = L.run(L.rings(R), [n])                     # a prompt in one call
    for i in range(b):
        close(whole[i], *L.oracle(i, n), dtype)
    short = coff * ratio                               # the smallest ring: one token a call, or several
    assert torch.equal(L.run(L.rings(short), [n]), whole)
    assert torch.equal(L.run(L.rings(short), [1] * n), whole)
    cuts = [5, 1, 2, n // 2 - 4, 3, n - n // 2 - 7] if n > 20 else [3, 1, n - 4]
    assert torch.equal(L.run(L.rings(short), cuts), whole)
    assert torch.equal(L.run(L.rings(short + 3), cuts), whole)


def test_rings_hold_the_newest_rows():
    L = Layer(37, 2, 29, 64, 4, 2, "d", BF)
    for R, sizes in ((8, [29]), (8, [1] * 29), (13, [20, 9]), (40, [29])):
        kr, sr = L.rings(R)
        L.run((kr, sr), sizes)
        held = list(range(max(0, 29 - R), 29))
        slots = [p % R for p in held]
        assert torch.equal(kr[:, slots], L.kv[:, held]) and torch.equal(sr[:, slots], L.score[:, held])
        rest = [r for r in range(R) if r not in slots]
        assert bool(kr[:, rest].isnan().all()) and bool(sr[:, rest].isnan().all())


def test_ragged_batches_padding_and_rows_left_alone():
    """Lengths of 0, 1, shorter than the call, in the middle of a block, at its end; NaN in padding."""
    L = Layer(41, 8, 40, 128, 4, 2, "d", BF)
    s = 6
    lens = [0, 1, 5, 6, 7, 12, 39, 40]
    rings = L.rings(2 * 4 - 1 + s)
    kv, score = torch.full((8, s, 128), float("nan"), dtype=BF, device="cuda"), torch.full((8, s, 128), float("nan"), dtype=BF, device="cuda")
    want = []
    for i, n in enumerate(lens):
        for p in range(max(0, n - s)):
            rings[0][i, p % 13], rings[1][i, p % 13] = L.kv[i, p], L.score[i, p]
        k = min(n, s)
        if k:
            kv[i, s - k:], score[i, s - k:] = L.kv[i, n - k:n], L.score[i, n - k:n]
        want.append(L.oracle(i, n))
    before = [t.clone() for t in rings]
    out = torch.full((8, 2, 128), 9.0, dtype=BF, device="cuda")
    got, first, counts = rows.csa_compress_decode(kv, score, *rings, ints(lens), 4, 2, L.kind, L.weight, None, EPS, L.rope, out=out)
    assert got is out
    for i, n in enumerate(lens):
        j, k = max(0, n - s) // 4, n // 4 - max(0, n - s) // 4
        assert (first[i].item(), counts[i].item()) == (j, k)
        close(out[i, :k], want[i][0][j:j + k], want[i][1][j:j + k], BF)
        assert bool((out[i, k:] == 9).all())
        new = [p % 13 for p in range(max(0, n - s), n)]
        for ring, was, src in zip(rings, before, (L.kv, L.score)):
            assert torch.equal(ring[i, new], src[i, max(0, n - s):n])
            same = [r for r in range(13) if r not in new]
            assert torch.equal(ring[i, same].view(torch.int16), was[i, same].view(torch.int16))


def test_negative_lengths_are_recorded():
    L = Layer(43, 2, 8, 64, 4, 1, "d", BF)
    rings = L.rings(8)
    _, first, counts = L.call(rings, 0, 4, lens=ints([-3, 4]))
    assert first.tolist() == [0, 0] and counts.tolist() == [0, 1]
    assert csa.csa_get_device_status(with_site=True) == (6, 0x72)
    assert bool(rings[0][0].isnan().all())


def test_drafts_taken_back():
    """Three draft tokens a step, of which some are dropped and replaced."""
    L = Layer(47, 2, 61, 128, 4, 2, "d", BF)
    other = Layer(48, 2, 61, 128, 4, 2, "d", BF)
    want = L.run(L.rings(100), [61])
    rings = L.rings(2 * 4 - 1 + 3)
    got, at = torch.zeros_like(want), 0
    keep = [1, 2, 3, 1, 1, 3, 2]
    step = 0
    while at + 3 <= 61:
        k = keep[step % len(keep)]
        kv, score = other.kv[:, at:at + 3].clone(), other.score[:, at:at + 3].clone()
        kv[:, :k], score[:, :k] = L.kv[:, at:at + k], L.score[:, at:at + k]
        out, _, _ = rows.csa_compress_decode(kv, score, *rings, ints([at + 3] * 2), 4, 2, L.kind, L.weight, None, EPS, L.rope)
        j0, j1 = at // 4, (at + k) // 4
        got[:, j0:j1] = out[:, :j1 - j0]
        at += k
        step += 1
    assert torch.equal(got[:, :at // 4], want[:, :at // 4])


@pytest.mark.parametrize("ratio,coff", [(4, 1), (4, 2), (128, 1)])
def test_rows_of_the_whole_sequence_calls(ratio, coff):
    """csa_compress_norm_rope and csa_compress_overlap give the same rows, up to fp32 rounding before the casts: each side is
    within the oracle's bound."""
    L = Layer(53, 2, 260, 128, ratio, coff, "d", BF, orc.RMS if coff == 1 else 0, 64 if coff == 1 else 0)
    got = L.run(L.rings(coff * ratio), [101, 27, 132])
    if coff == 1:
        ref = csa.csa_compress_norm_rope(L.kv, L.score, ratio, L.weight, EPS, 64, 40000.0)
    else:
        ref = csa.csa_compress_overlap(L.kv, L.score, ratio, coff)
    for i in range(2):
        want, err = L.oracle(i, 260)
        step = orc.STEP["bf16"] * (np.abs(want) + err)
        assert (np.abs(f64(got[i]) - f64(ref[i])) <= 2 * (err + step) + 1e-37).all()


def test_scores_of_minus_infinity():
    """Masked tokens have no weight, also at the start of a block."""
    L = Layer(59, 1, 24, 64, 8, 1, 1, F32, 0, 0)
    L.score[0, [0, 1, 9, 23]] = float("-inf")
    got = L.run(L.rings(8), [24])
    z = f64(L.score[0])
    for j in range(3):
        t = slice(8 * j, 8 * j + 8)
        w = np.exp(z[t] - z[t].max())
        want = (w * f64(L.kv[0, t])).sum(0) / w.sum()
        assert np.abs(f64(got[0, j]) - want).max() <= 64 * orc.U * np.abs(f64(L.kv)).max()


@pytest.mark.parametrize("ratio,coff", [(8, 1), (8, 2), (128, 1)])
def test_a_block_of_minus_infinities(ratio, coff):
    """A channel whose scores are all -inf has no weights: NaN there, and nowhere else."""
    n = 3 * ratio
    L = Layer(89, 2, n, 64, ratio, coff, "d", F32, 0, 0)
    want = L.run(L.rings(coff * ratio), [n])
    L.score[1, :2 * ratio, 5] = float("-inf")
    got = L.run(L.rings(coff * ratio), [n])
    none = torch.zeros_like(got, dtype=torch.bool)
    none[1, :2, 5] = True
    assert torch.equal(got.isnan(), none)
    keep = ~none
    keep[1, :, 5] = False
    assert torch.equal(got[keep], want[keep])


def test_strided_inputs_and_streams():
    L = Layer(61, 3, 30, 64, 4, 2, "d", BF)
    want = L.run(L.rings(8), [30])
    fused = torch.cat((L.kv, L.score), -1)
    out = torch.zeros(3, 10, 64, dtype=BF, device="cuda")
    rings = L.rings(8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, first, counts = rows.csa_compress_decode(fused[..., :64], fused[..., 64:], *rings, ints([30] * 3), 4, 2, L.kind, L.weight, None, EPS,
                                                  L.rope, out=out[:, :8], stream=side)
    side.synchronize()
    assert torch.equal(out[:, :7], want) and not out[:, 7:].any()
    one = Layer(61, 1, 30, 64, 4, 2, 1, F32)
    wide = torch.randn(1, 30, 5, device="cuda")
    wide[..., 3:4] = one.score
    a = one.run(one.rings(8), [30])
    b, _, _ = rows.csa_compress_decode(one.kv, wide[..., 3:4], *one.rings(8), ints([30]), 4, 2, one.kind, one.weight, None, EPS, one.rope)
    assert torch.equal(a, b[:, :7])


def test_rings_beyond_32_bits():
    """Sequences whose rings start behind 2^31 elements."""
    L = Layer(73, 5, 24, 512, 4, 2, "d", BF, orc.RMS, 64)
    want = L.run(L.rings(8), [24])
    rings = tuple(torch.full((5, (1 << 20) + 7, 512), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    assert torch.equal(L.run(rings, [9, 1, 1, 1, 12]), want)
    assert torch.equal(rings[0][:, :24], L.kv) and torch.equal(rings[1][:, :24], L.score)


def test_no_new_tokens():
    L = Layer(83, 3, 8, 64, 4, 2, "d", BF)
    rings = L.rings(8)
    L.run(rings, [8])
    held = [t.clone() for t in rings]
    torch.full((3,), 77, dtype=I32, device="cuda")     # (what the next tensors of this size would find)
    torch.full((3,), 77, dtype=I32, device="cuda")
    out, first, counts = L.call(rings, 8, 0, lens=ints([8, 3, 0]))
    assert out.shape == (3, 0, 64) and first.tolist() == counts.tolist() == [0] * 3
    mine = [ints([5] * 3), ints([6] * 3)]
    L.call(rings, 8, 0, lens=ints([8, 3, 0]), first=mine[0], counts=mine[1])
    assert mine[0].tolist() == [5] * 3 and mine[1].tolist() == [6] * 3
    assert all(torch.equal(a, b) for a, b in zip(rings, held))


@pytest.mark.parametrize("d,ratio,coff,R,small", [(64, 4, 2, 8, 23), (64, 4, 1, 8, 31), (512, 1, 1, 8, 15), (64, 1, 2, 4, 11)])
def test_the_longest_sequences(d, ratio, coff, R, small):
    """Sequences that end at 2^31 - 1: the same rows, bit for bit, as of a short one that ends at the same place of its block and
    of its ring (nothing turned: the rotation alone would tell them apart)."""
    top = 2 ** 31 - 1
    assert top % R == small % R and top % ratio == small % ratio
    for s in (1, 2, 5):
        L = Layer(79, 2, small, d, ratio, coff, "d", BF, orc.RMS, 0)
        rings = L.rings(R)
        L.run(rings, [small - s])
        far = tuple(t.clone() for t in rings)
        out, first, counts = L.call(rings, small - s, s)
        got, far_first, far_counts = L.call(far, small - s, s, lens=ints([top] * 2))
        k = top // ratio - (top - s) // ratio
        assert far_first.tolist() == [(top - s) // ratio] * 2 and far_counts.tolist() == counts.tolist() == [k] * 2
        assert torch.equal(got[:, :k], out[:, :k])
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(rings, far))


def test_the_binding_refuses():
    L = Layer(67, 2, 8, 64, 4, 1, "d", BF)
    kr, sr = L.rings(8)
    lens = ints([8, 8])
    ok = dict(kv=L.kv, score=L.score, kv_ring=kr, score_ring=sr, seq_lens=lens, ratio=4)
    rows.csa_compress_decode(**ok)
    for bad in (dict(score=L.score.float()), dict(score=L.score[:, :4]), dict(kv_ring=kr[:, :, :32]), dict(score_ring=sr[:1]),
                dict(seq_lens=lens.long()), dict(seq_lens=lens.cpu()), dict(kv=L.kv.transpose(1, 2)), dict(kv_ring=kr[:, :3].contiguous()),
                dict(ratio=0), dict(coff=3), dict(coff=0), dict(kind=5), dict(rope="x"), dict(out=torch.zeros(2, 3, 64, dtype=BF, device="cuda")),
                dict(out=torch.zeros(2, 2, 64, device="cuda")), dict(first=torch.zeros(2, device="cuda")), dict(weight=torch.ones(8, device="cuda"), kind=1)):
        with pytest.raises((ValueError, TypeError, csa.CSAError)):
            rows.csa_compress_decode(**{**ok, **bad})
            pytest.fail(f"{sorted(bad)} was not refused")


@pytest.mark.parametrize("bits", [4, 8])
def test_a_captured_decode_step_matches_the_whole_sequence_calls(bits):
    """One layer whose rows are normalised and turned.  A step, captured once, does everything for the next token of every
    sequence from lengths on the device: q and the raw row normed and turned, both written, blocks and index keys pooled as they
    complete and written, select, attend, o turned back.  The whole-sequence calls on the same rows (read back from the cache)
    give the same selection, and the same output up to both sides' rounding."""
    g = torch.Generator().manual_seed(71)
    b, n, H, d, H_I, d_I, ratio, coff, window, topk, page = 2, 75, 32, 128, 64, 128, 4, 2, 20, 6, 16
    draw = lambda *shape: torch.randn(*shape, generator=g).to(BF).cuda()  # noqa: E731
    q, kv, q_I = draw(b, n, H, d), draw(b, n, d), draw(b, n, H_I, d_I)
    ckv, cscore, ikv, iscore = draw(b, n, d), draw(b, n, d), draw(b, n, d_I), draw(b, n, d_I)
    w = (torch.randn(b, n, H_I, generator=g) / 2).cuda()
    sink = torch.randn(H, generator=g).cuda()
    nw, cw, iw, ib = ((0.5 + torch.rand(d, generator=g)).cuda() for _ in range(4))
    rope = rows.CsaRope(rows.csa_rope_turns(rows.csa_rope_freqs(64, 10000.0)), 64)
    crope = rows.CsaRope(rows.csa_rope_turns(rows.csa_rope_freqs(64, 40000.0)), 64)
    irope = rows.CsaRope(rows.csa_rope_turns(rows.csa_rope_freqs(64, 40000.0)), 0, "half")
    n_c, scale = n // ratio, d ** -0.5
    P_all, P_cmp = -(-n // page), -(-n_c // page)
    raw_t = torch.arange(b * P_all, dtype=I32, device="cuda").view(b, P_all)
    cmp_t = (torch.arange(b * P_cmp, dtype=I32, device="cuda") + b * P_all).view(b, P_cmp)
    key_t = torch.arange(b * P_cmp, dtype=I32, device="cuda").view(b, P_cmp)
    cache = torch.full((b * (P_all + P_cmp), serve.csa_cache_page_bytes(page, d, bits)), 0xFF, dtype=U8, device="cuda")
    icache = torch.full((b * P_cmp, serve.csa_cache_page_bytes(page, d_I, bits)), 0xFF, dtype=U8, device="cuda")
    rings = [torch.zeros(b, coff * ratio, c, dtype=BF, device="cuda") for c in (d, d, d_I, d_I)]
    lens = torch.zeros(b, dtype=I32, device="cuda")
    now = [t[:, :1].clone() for t in (q, kv, q_I, ckv, cscore, ikv, iscore, w)]

    def step():
        tq, tkv, tq_I, tc, ts, ti, tis, tw = now
        lens.add_(1)
        at = lens - 1
        pos = at[:, None]
        y = rows.csa_norm_rope(tq, rows.CSA_NORM_RMS, rope, pos, nw, None, EPS)
        r = rows.csa_norm_rope(tkv, rows.CSA_NORM_RMS, rope, pos, nw, None, EPS)
        serve.csa_cache_write(r, cache, raw_t, at, page, bits)
        out, first, counts = rows.csa_compress_decode(tc, ts, rings[0], rings[1], lens, ratio, coff, rows.CSA_NORM_RMS, cw, None, EPS, crope)
        serve.csa_cache_write(out, cache, cmp_t, first, page, bits, counts=counts)
        keys, first, counts = rows.csa_compress_decode(ti, tis, rings[2], rings[3], lens, ratio, coff, rows.CSA_NORM_LAYER, iw, ib, EPS, irope)
        serve.csa_cache_write(keys, icache, key_t, first, page, bits, counts=counts)
        idx = serve.csa_indexer_topk_decode(rows.csa_rope(tq_I, irope, pos), icache, key_t, tw, lens, topk, ratio, page, bits)
        o, lse = serve.csa_attn_decode(y, cache, raw_t, cmp_t, idx, sink, lens, scale, ratio, window, page, bits)
        return y, idx, o, lse, rows.csa_rope(o, rope, pos, inverse=True)

    step()                                             # outside of a graph first; taken back below
    lens.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    Y, O, Z = (torch.zeros(b, n, H, d, dtype=BF, device="cuda") for _ in range(3))
    I, L = torch.full((b, n, topk), -1, dtype=I32, device="cuda"), torch.zeros(b, n, H, device="cuda")
    lens.zero_()
    for t in range(n):
        for x, src in zip(now, (q, kv, q_I, ckv, cscore, ikv, iscore, w)):
            x.copy_(src[:, t:t + 1])
        graph.replay()
        for x, y in zip((Y, I, O, L, Z), got):
            x[:, t:t + 1] = y
    assert lens.tolist() == [n] * b
    zero = torch.zeros(b, dtype=I32, device="cuda")
    # what the steps made, by calls on the whole sequence: bit for bit
    assert torch.equal(Y, rows.csa_norm_rope(q, rows.CSA_NORM_RMS, rope, None, nw, None, EPS))
    kv_full = torch.empty(b, n + n_c, d, dtype=BF, device="cuda")
    serve.csa_cache_read(cache, raw_t, zero, kv_full[:, :n], page, bits)
    serve.csa_cache_read(cache, cmp_t, zero, kv_full[:, n:], page, bits)
    k_I = serve.csa_cache_read(icache, key_t, zero, torch.empty(b, n_c, d_I, dtype=BF, device="cuda"), page, bits)
    again = torch.full_like(cache, 0xFF)
    iagain = torch.full_like(icache, 0xFF)
    serve.csa_cache_write(rows.csa_norm_rope(kv, rows.CSA_NORM_RMS, rope, None, nw, None, EPS), again, raw_t, zero, page, bits)
    full = [torch.zeros(b, coff * ratio, c, dtype=BF, device="cuda") for c in (d, d, d_I, d_I)]
    all_lens = zero + n
    out, first, counts = rows.csa_compress_decode(ckv, cscore, full[0], full[1], all_lens, ratio, coff, rows.CSA_NORM_RMS, cw, None, EPS, crope)
    serve.csa_cache_write(out, again, cmp_t, first, page, bits, counts=counts)
    out, first, counts = rows.csa_compress_decode(ikv, iscore, full[2], full[3], all_lens, ratio, coff, rows.CSA_NORM_LAYER, iw, ib, EPS, irope)
    serve.csa_cache_write(out, iagain, key_t, first, page, bits, counts=counts)
    assert torch.equal(cache, again) and torch.equal(icache, iagain)
    assert all(torch.equal(p, r) for p, r in zip(rings, full))
    ref_idx = csa.csa_indexer_topk(rows.csa_rope(q_I, irope), k_I, w, topk, ratio)
    assert torch.equal(I, ref_idx)
    ref_o, ref_l = csa.csa_attn_fwd(Y, kv_full, I, sink, scale, ratio, window)
    # each side: probabilities and their sum rounded to bf16 (2 x 2^-8) and o rounded once (2^-8), of at most the largest |v|
    top = kv_full.float().abs().max().item()
    assert (O.float() - ref_o.float()).abs().max().item() <= 2 * 3 * 2.0 ** -8 * top
    # logits of at most 1.5^2 |x||y| d scale = 25, summed in 16 steps on each side
    assert (L - ref_l).abs().max().item() <= 25 * 16 * 2 * 2.0 ** -22
    assert torch.equal(Z, rows.csa_rope(O, rope, None, inverse=True))


LOWEST = "lowest of the type"
MASKED = [
    # dtype, ratio, coff, d, masked tokens, tokens
    (BF, 128, 1, 512, range(64), 128),                 # whole slices, and a thread's first group
    (BF, 128, 1, 128, range(120), 128),                # all but the last slice's last tokens
    (BF, 128, 1, 128, range(8, 256), 256),             # most of a block; a block of nothing else
    (F32, 4, 2, 64, range(4), 12),                     # the block before a sequence's first real one
    (F32, 4, 1, 64, range(8), 12),                     # blocks of nothing else
    (F32, 8, 1, 72, [0, 1, 2, 3, 9, 15, 16, 23], 24),  # a thread's first group; single tokens
    (BF, 4, 2, 512, [0, 1, 2, 3, 5, 8, 11], 16),
    (F32, 128, 2, 512, range(100, 260), 384),
]


@pytest.mark.parametrize("value", [-1e4, -1e10, -1e20, -1e30, LOWEST])
@pytest.mark.parametrize("case", MASKED, ids=str)
def test_scores_masked_by_a_finite_value(case, value):
    """Tokens with scores far below the others have no weight, wherever a block has them; a block of nothing else is their mean."""
    dtype, ratio, coff, d, masked, n = case
    for sw in ("d", 1):
        L = Layer(97, 2, n, d, ratio, coff, sw, dtype, 0, 0)
        L.score[1, list(masked)] = torch.finfo(dtype).min if value is LOWEST else value
        got = L.run(L.rings(coff * ratio), [n])
        assert torch.equal(L.run(L.rings(coff * ratio), [1] * n), got)
        for i in range(2):
            close(got[i], *L.oracle(i, n), dtype)
        # the whole-sequence call, where a window has a token that is not masked
        whole = csa.csa_compress_overlap(L.kv, L.score, ratio, coff)
        want, err = L.oracle(1, n)
        off = np.abs(f64(got[1]) - f64(whole[1])) - 2 * (err + orc.STEP[NAME[dtype]] * (np.abs(want) + err)) - 1e-37
        for j in range(n // ratio):
            if not set(range(max(0, (j + 1 - coff) * ratio), (j + 1) * ratio)) <= set(masked):
                assert (off[j] <= 0).all(), j


@pytest.mark.parametrize("ratio,coff,d", [(4, 2, 64), (8, 1, 512), (128, 1, 128), (100, 2, 80)])
@pytest.mark.parametrize("offset", [0.0, 300.0, -3000.0, 30000.0, 1e9, -1e30])
def test_a_common_offset_of_the_scores(ratio, coff, d, offset):
    """The softmax does not depend on it; what fp32 leaves of the scores is what both sides are given."""
    n = 3 * ratio
    L = Layer(101, 1, n, d, ratio, coff, "d", F32, 0, 0)
    L.score += offset
    close(L.run(L.rings(coff * ratio), [n])[0], *L.oracle(0, n), F32)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_token_far_above_the_others(dtype):
    """It alone has weight: its row, to the bit, also where the difference of two scores leaves the type."""
    for ratio, coff, top in ((4, 1, 1e4), (16, 1, 1e30), (128, 1, torch.finfo(dtype).max), (4, 2, torch.finfo(dtype).max)):
        L = Layer(103, 1, 2 * ratio, 64, ratio, coff, "d", dtype, 0, 0)
        for at in (0, ratio // 2, ratio - 1):
            L.score.clamp_(-4, 4)
            L.score[0, ratio + at] = top
            L.score[0, ratio + (at + 1) % ratio] = torch.finfo(dtype).min
            assert torch.equal(L.run(L.rings(coff * ratio), [2 * ratio])[0, 1], L.kv[0, ratio + at])


@pytest.mark.parametrize("s_q", [2 ** 31 - 1, 2 ** 31 - 300])
def test_the_longest_call(s_q):
    """As many new tokens as there can be, each a block: every row of out is its token's."""
    d = 8
    row = torch.arange(1, d + 1, device="cuda").to(BF).view(1, 1, d)
    kv, score = row.expand(1, s_q, d), torch.zeros(1, 1, 1, dtype=BF, device="cuda").expand(1, s_q, 1)
    kr, sr = torch.zeros(1, 4, d, dtype=BF, device="cuda"), torch.zeros(1, 4, 1, dtype=BF, device="cuda")
    out, first, counts = rows.csa_compress_decode(kv, score, kr, sr, ints([s_q]), 1)
    assert out.shape == (1, s_q, d) and first.tolist() == [0] and counts.tolist() == [s_q]
    for i in range(0, s_q, 1 << 28):
        assert bool((out[:, i:i + (1 << 28)] == row).all()), i
    assert bool((kr == row).all())
    del out
    torch.cuda.empty_cache()
