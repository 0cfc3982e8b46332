"""The serving calls on the GPU against the fp64 oracle: the quantised paged
cache (byte for byte), the single-token indexer (exact sets) and the
single-token attention (bounds derived below), their streams and graphs, and a
decode loop that uses all of them together."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_sum_gb300 import csa, serve
from oracle import serve_oracle as orc

pytestmark = pytest.mark.gpu

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
DEVICE_CHECK, SITE_PAGE, SITE_RANGE = 6, 0x71, 0x72
POISON = 0xFF        # NaN codes and an infinite scale: no row that is not visible may matter


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from compressed_sparse_attention_sum_gb300 import build
    build.build()
    serve.load_library()
    csa.csa_get_device_status()
    yield
    assert csa.csa_get_device_status() == 0


def dev(x, dtype=None):
    t = x if isinstance(x, torch.Tensor) else torch.as_tensor(np.asarray(x))
    return t.to(dtype) .cuda() if dtype is not None else t.cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def empty_cache(n_pages, page, d, bits, fill=POISON):
    return torch.full((n_pages, serve.csa_cache_page_bytes(page, d, bits)), fill, dtype=U8,
                      device="cuda")


def tables(rng, b, *widths, spare=2):
    """Page tables over one pool in random order; returns (n_pages, tables)."""
    total = b * sum(widths)
    ids = rng.permutation(total + spare)[:total]
    out, at = [], 0
    for w in widths:
        out.append(ids[at:at + b * w].reshape(b, w).astype(np.int32))
        at += b * w
    return total + spare, out


# ------------------------------------------------------------------ cache

def special_rows(rng, shape, dtype):
    """N(0, 1) rows with rounding ties, exact group maxima, zeros and extreme magnitudes."""
    x = rng.standard_normal(shape).astype(np.float32)
    flat = x.reshape(-1, 32)
    n = len(flat)
    flat[0 % n, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    flat[0 % n, 8:] = np.clip(flat[0 % n, 8:], -6, 6)
    flat[1 % n] = 0.0
    flat[2 % n] *= np.float32(2.0 ** 100)
    flat[3 % n] *= np.float32(2.0 ** -118)       # below the smallest scale
    flat[4 % n, 3] = -448.0
    flat[5 % n, 0] = np.float32(-6.0000005)
    flat[6 % n] = -0.0
    return torch.from_numpy(x).to(dtype)


CACHE_CASES = [
    # bits, dtype, d, page, b, s, P, pos0 (first), ragged
    (4, BF, 128, 64, 3, 5, 2, 61, False),
    (4, F32, 32, 16, 2, 17, 2, 0, True),
    (4, BF, 512, 16, 2, 33, 4, 7, True),
    (8, BF, 128, 48, 3, 50, 2, 40, True),
    (8, F32, 64, 16, 1, 1, 1, 1000003, False),
    (8, F32, 320, 16, 2, 40, 1, 11, False),      # more rows than the ring holds
    (4, BF, 96, 16, 4, 70, 2, 2147483000, True),
]


@pytest.mark.parametrize("case", CACHE_CASES, ids=lambda c: f"{c[0]}bit_d{c[2]}_s{c[5]}_P{c[6]}")
def test_write_bytes_and_read_back(case):
    bits, dtype, d, page, b, s, P, first, ragged = case
    rng = np.random.default_rng(d + s)
    n_pages, (table,) = tables(rng, b, P)
    pos0 = np.array([first + 3 * i for i in range(b)], np.int32)
    counts = np.array([s] + [int(rng.integers(0, s + 1)) for _ in range(b - 1)] if ragged else [s] * b)
    if ragged:
        counts[-1] = 0 if b > 1 else s
    x = special_rows(rng, (b, s, d), dtype)
    # rows and batches at strides of their own, the gaps holding NaN
    pitch, gap = d + 16, 24
    buf = torch.full((b, s * pitch + gap), float("nan"), dtype=dtype, device="cuda")
    xs = buf[:, :s * pitch].unflatten(1, (s, pitch))[..., :d]
    xs.copy_(x)
    cache = empty_cache(n_pages, page, d, bits)
    before = cache.cpu().numpy()
    got = serve.csa_cache_write(xs, cache, dev(table), dev(pos0), page, bits,
                                counts=dev(counts, I32) if ragged else None)
    assert got is cache
    want = orc.write(before, f64(x), table, pos0, counts, page, bits)
    assert np.array_equal(cache.cpu().numpy(), want)

    # read the newest rows that the ring still holds
    ring = P * page
    start = np.array([max(0, c - ring) for c in counts])
    n = min(s, ring)
    left = np.minimum(counts - start, n)
    for out_dtype in (BF, F32):
        out = torch.full((b, n, d + 8), 7.0, dtype=out_dtype, device="cuda")
        serve.csa_cache_read(cache, dev(table), dev((pos0 + start).astype(np.int32)), out[..., :d], page,
                             bits, counts=dev(left, I32))
        got = f64(out)
        assert (got[..., d:] == 7.0).all()
        for i in range(b):
            for r in range(n):
                want_row = (orc.held_rows(f64(x)[i, start[i] + r][None], bits)[0] if r < left[i]
                            else np.full(d, 7.0))
                assert np.array_equal(got[i, r, :d], want_row), (i, r)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 96, 512])
def test_long_ranges_equal_short_ones(bits, d):
    """The kernels of long ranges (several rows a thread, 8 or 16 channels by
    alignment) write and read what the same rows in short calls do."""
    rng = np.random.default_rng(d)
    b, page, s = 2, 48, 2500 * 256 // (d // 8) // 2 + 77
    P = -(-s // page) + 1
    n_pages, (table,) = tables(rng, b, P)
    table, pos0 = dev(table), dev(np.array([5, 41], np.int32))
    counts = dev(np.array([s, s - 130], np.int32))
    g = torch.Generator(device="cuda").manual_seed(d)
    buf = torch.randn(b, s + 1, d + 8, generator=g, device="cuda").to(BF) * 3
    want = empty_cache(n_pages, page, d, bits)
    x = buf[:, :s, :d].contiguous()
    for at in range(0, s, 999):
        n = min(999, s - at)
        serve.csa_cache_write(x[:, at:at + n], want, table, pos0 + at, page, bits,
                              counts=(counts - at).clamp(min=0, max=n))
    for rows in (x, buf[:, :s, :d], x.float()):        # 32-byte boundaries, 16-byte ones, fp32
        cache = empty_cache(n_pages, page, d, bits)
        serve.csa_cache_write(rows, cache, table, pos0, page, bits, counts=counts)
        assert torch.equal(cache, want)
    ref = torch.full((b, s, d), 7.0, dtype=BF, device="cuda")
    for at in range(0, s, 999):
        n = min(999, s - at)
        serve.csa_cache_read(want, table, pos0 + at, ref[:, at:at + n], page, bits,
                             counts=(counts - at).clamp(min=0, max=n))
    assert bool((ref[1, s - 130:] == 7.0).all())
    wide = torch.full((b, s, d), 7.0, dtype=BF, device="cuda")
    odd = torch.full((b, s, d + 8), 7.0, dtype=BF, device="cuda")
    single = torch.full((b, s, d), 7.0, device="cuda")
    for out in (wide, odd[..., :d], single):
        serve.csa_cache_read(want, table, pos0, out, page, bits, counts=counts)
        assert torch.equal(out.to(BF), ref)
    assert bool((odd[..., d:] == 7.0).all())


@pytest.mark.parametrize("bits,top", [(4, 1.5 * 2.0 ** 127), (8, 1.75 * 2.0 ** 127)])
def test_the_largest_magnitudes_saturate(bits, top):
    """Groups up to the end of fp32: the scale stops where its largest code is a
    bf16 value, and what lies beyond is that value."""
    x = torch.zeros(1, 4, 64)
    x[0, 0, 0], x[0, 0, 40], x[0, 1, 3] = 3.4e38, -3.4e38, 2.0 ** 127
    x[0, 2, 5], x[0, 2, 63] = 1.5 * 2.0 ** 127, -1.25 * 2.0 ** 126
    x[0, 3, 0], x[0, 3, 1] = float("inf"), 2.0 ** 126
    cache = empty_cache(1, 16, 64, bits)
    out = torch.empty(1, 4, 64, device="cuda")
    args = (dev([[0]], I32), dev([0], I32))
    serve.csa_cache_write(x.cuda(), cache, *args, 16, bits)
    serve.csa_cache_read(cache, *args, out, 16, bits)
    got = f64(out)[0]
    assert np.array_equal(got[:3], orc.held_rows(x[0, :3].numpy(), bits))
    assert got[0, 0] == top and got[0, 40] == -top and got[3, 0] == top and got[3, 1] == 2.0 ** 126


def test_bad_pages_and_counts_are_skipped_and_recorded():
    bits, d, page = 4, 64, 16
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((3, 20, d))).to(BF)
    table = np.array([[0, 5], [2, -1], [4, 3]], np.int32)          # 6 pages: 5 is inside, -1 and 99 are not
    table_bad = table.copy()
    table_bad[0, 1] = 99
    cache = empty_cache(6, page, d, bits)
    before = cache.cpu().numpy()
    zeros = dev(np.zeros(3, np.int32))
    serve.csa_cache_write(x.cuda(), cache, dev(table_bad), zeros, page, bits)
    assert csa.csa_get_device_status(with_site=True) == (DEVICE_CHECK, SITE_PAGE)
    want = orc.write(before, f64(x), table, [0, 0, 0], [16, 16, 20], page, bits)
    assert np.array_equal(cache.cpu().numpy(), want)
    out = torch.full((3, 20, d), 7.0, dtype=BF, device="cuda")
    serve.csa_cache_read(cache, dev(table_bad), zeros, out, page, bits)
    assert csa.csa_get_device_status(with_site=True) == (DEVICE_CHECK, SITE_PAGE)
    held = orc.held_rows(f64(x), bits)
    held[:2, 16:] = 0.0                                            # rows of the bad pages
    assert np.array_equal(f64(out), held)
    # counts outside [0, s] are clamped, a negative position moves nothing
    cache = empty_cache(6, page, d, bits)
    table[1, 1] = 1
    serve.csa_cache_write(x.cuda(), cache, dev(table), dev(np.array([0, -4, 2], np.int32)), page, bits,
                          counts=dev(np.array([-3, 20, 99], np.int32)))
    assert csa.csa_get_device_status(with_site=True) == (DEVICE_CHECK, SITE_RANGE)
    want = orc.write(before, f64(x), table, [0, 0, 2], [0, 0, 20], page, bits)
    assert np.array_equal(cache.cpu().numpy(), want)


def test_offsets_beyond_32_bits():
    """A cache of 5.1 GB: pages whose byte offsets pass 2^32, for all four calls."""
    bits, d, page = 8, 512, 64
    page_bytes = serve.csa_cache_page_bytes(page, d, bits)
    n_pages = (5 << 30) // page_bytes + 1
    cache = torch.empty(n_pages, page_bytes, dtype=U8, device="cuda")
    rng = np.random.default_rng(5)
    raw_t, cmp_t = [[n_pages - 1, n_pages - 2]], [[n_pages - 5, 3]]
    raw = torch.from_numpy(rng.standard_normal((1, 100, d))).to(BF)
    cmp = torch.from_numpy(rng.standard_normal((1, 100, d))).to(BF)
    zero = dev(np.zeros(1, np.int32))
    for x, t in ((raw, raw_t), (cmp, cmp_t)):
        serve.csa_cache_write(x.cuda(), cache, dev(t, I32), zero, page, bits)
        out = torch.zeros(1, 100, d, dtype=F32, device="cuda")
        serve.csa_cache_read(cache, dev(t, I32), zero, out, page, bits)
        assert np.array_equal(f64(out), orc.held_rows(f64(x), bits))
    q = torch.from_numpy(rng.standard_normal((1, 1, 64, d))).to(BF)
    lens = dev(np.array([100], np.int32))
    o, lse = serve.csa_attn_decode(q.cuda(), cache, dev(raw_t, I32), dev(cmp_t, I32), None, None, lens,
                                   d ** -0.5, 1, 33, page, bits)
    r, c = orc.held_rows(f64(raw[0]), bits), orc.held_rows(f64(cmp[0]), bits)
    check_row(o[0, 0], lse[0, 0], f64(q)[0, 0], lambda p: r[p], lambda j: c[j], None, None, d ** -0.5, 99,
              1, 33, BF)
    del cache
    d = 128
    page_bytes = serve.csa_cache_page_bytes(page, d, bits)
    n_pages = (5 << 30) // page_bytes + 1
    cache = torch.empty(n_pages, page_bytes, dtype=U8, device="cuda")
    keys = torch.from_numpy(rng.standard_normal((1, 100, d))).to(BF)
    serve.csa_cache_write(keys.cuda(), cache, dev(cmp_t, I32) * 0 + dev([[n_pages - 1, n_pages - 4]], I32),
                          zero, page, bits)
    qi = torch.from_numpy(rng.standard_normal((1, 1, 64, d))).to(BF)
    w = torch.from_numpy(rng.standard_normal((1, 1, 64))).float()
    got = serve.csa_indexer_topk_decode(qi.cuda(), cache, dev([[n_pages - 1, n_pages - 4]], I32), w.cuda(),
                                        lens, 20, 1, page, bits)
    want = orc.index_row(f64(qi)[0, 0], f64(w)[0, 0], orc.held_rows(f64(keys[0]), bits), 99, 1, 20)
    assert np.array_equal(got.cpu().numpy()[0, 0], want)


# ---------------------------------------------------------------- indexer

def index_case(rng, b, s_q, H, d, ratio, lens, bits, page, dtype, keys=None):
    n = max(1, max(lens) // ratio)
    P = -(-n // page)
    n_pages, (table,) = tables(rng, b, P)
    if keys is None:
        keys = torch.from_numpy(rng.standard_normal((b, n, d))).to(BF)
    cache = empty_cache(n_pages, page, d, bits)
    serve.csa_cache_write(keys.cuda(), cache, dev(table), dev(np.zeros(b, np.int32)), page, bits)
    q = torch.from_numpy(rng.standard_normal((b, s_q, H, d))).to(dtype)
    w = torch.from_numpy(rng.standard_normal((b, s_q, H)) / 2).float()
    return cache, table, keys, q, w


def index_oracle(q, w, keys, lens, ratio, topk, bits):
    b, s_q = q.shape[:2]
    out = np.empty((b, s_q, topk), np.int64)
    for s in range(b):
        held = orc.held_rows(f64(keys[s]), bits)
        for i in range(s_q):
            out[s, i] = orc.index_row(f64(q)[s, i], f64(w)[s, i], held, lens[s] - s_q + i, ratio, topk)
    return out


INDEX_CASES = [
    # b, s_q, H, d, ratio, lens, topk, bits, page, dtype
    (1, 1, 64, 128, 4, [1200], 64, 4, 64, BF),
    (4, 1, 64, 128, 4, [0, 1, 3, 2051], 100, 4, 16, BF),
    (3, 2, 64, 128, 4, [1, 777, 1025], 33, 8, 48, BF),
    (2, 3, 32, 128, 1, [300, 129], 128, 4, 64, BF),
    (2, 1, 32, 64, 4, [1100, 515], 7, 8, 16, BF),
    (2, 2, 8, 64, 2, [700, 2], 1, 4, 32, BF),
    (1, 1, 3, 32, 4, [999], 17, 4, 16, BF),
    (1, 2, 70, 96, 4, [640], 50, 8, 16, BF),
    (2, 1, 4, 256, 4, [803, 90], 30, 8, 64, BF),
    (2, 1, 64, 128, 4, [900, 37], 50, 4, 64, F32),
    (1, 2, 5, 64, 3, [500], 20, 8, 16, F32),
    (1, 1, 16, 128, 128, [40000], 512, 4, 64, BF),      # topk above the visible blocks
    (1, 2, 70, 128, 4, [900], 40, 4, 16, BF),           # a query a CTA of 128 columns
    (2, 9, 8, 64, 2, [400, 5], 25, 8, 16, BF),          # nine queries: two groups of columns
    (1, 1, 128, 64, 1, [385], 100, 4, 128, BF),
]


@pytest.mark.parametrize("case", INDEX_CASES, ids=lambda c: f"b{c[0]}s{c[1]}H{c[2]}d{c[3]}k{c[6]}_{c[7]}bit")
def test_indexer_matches_oracle(case):
    b, s_q, H, d, ratio, lens, topk, bits, page, dtype = case
    rng = np.random.default_rng(H * d + topk)
    cache, table, keys, q, w = index_case(rng, b, s_q, H, d, ratio, lens, bits, page, dtype)
    got = serve.csa_indexer_topk_decode(q.cuda(), cache, dev(table), w.cuda(), dev(lens, I32), topk, ratio,
                                        page, bits)
    assert np.array_equal(got.cpu().numpy(), index_oracle(q, w, keys, lens, ratio, topk, bits))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kind", ["equal", "zero", "few", "swapped", "zero_w"])
def test_indexer_ties_go_to_the_lower_block(kind, bits):
    """Many blocks with exactly equal scores.  "swapped": a block's channels are
    exchanged where q has equal values, so that the exact scores are equal while
    sums of rounded numbers in channel order need not be."""
    rng = np.random.default_rng(11)
    H, d, ratio, page, n, topk = 64, 128, 1, 64, 700, 211
    base = rng.integers(-6, 7, (5, d)).astype(np.float64)
    q = np.repeat(rng.standard_normal((1, 1, H, d // 2)), 2, axis=-1)
    keys = base[rng.integers(0, 5, n)]
    if kind == "equal":
        keys = np.repeat(base[:1], n, 0)
    elif kind == "zero":
        keys = np.zeros((n, d))
    elif kind == "swapped":
        flip = rng.random((n, d // 2)) < 0.5
        pairs = np.repeat(base[:1], n, 0).reshape(n, d // 2, 2)
        keys = np.where(flip[..., None], pairs[..., ::-1], pairs).reshape(n, d)
    keys = torch.from_numpy(keys[None]).to(BF)
    cache, table, keys, _, w = index_case(rng, 1, 1, H, d, ratio, [n], bits, page, BF, keys=keys)
    q = torch.from_numpy(q).to(BF)
    if kind == "zero_w":
        w = w * 0
    got = serve.csa_indexer_topk_decode(q.cuda(), cache, dev(table), w.cuda(), dev([n], I32), topk, ratio,
                                        page, bits).cpu().numpy()[0, 0]
    held = orc.held_rows(f64(keys[0]), bits)
    if kind == "few":
        want = orc.index_row(f64(q)[0, 0], f64(w)[0, 0], held, n - 1, ratio, topk)
    else:
        want = np.arange(topk)
    assert np.array_equal(got, want)


def test_indexer_scores_closer_than_fp32():
    """Blocks whose exact scores differ by far less than fp32 resolves: two
    large channels cancel, a small third one decides."""
    rng = np.random.default_rng(12)
    n, d, H, topk = 300, 128, 32, 40
    keys = np.zeros((n, d))
    keys[:, 0], keys[:, 32] = 6.0, -6.0
    keys[:, 64] = 6.0                                   # the group's scale is 1
    tiny = rng.choice([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0], n)
    keys[:, 65] = tiny
    keys = torch.from_numpy(keys[None]).to(BF)
    q = np.zeros((1, 1, H, d))
    q[..., 0], q[..., 32] = 2.0 ** 20, 2.0 ** 20
    q[..., 64], q[..., 65] = 1.0, 2.0 ** -12
    cache, table, keys, _, w = index_case(rng, 1, 1, H, d, 1, [n], 4, 64, BF, keys=keys)
    w = w.abs() + 0.1
    got = serve.csa_indexer_topk_decode(torch.from_numpy(q).to(BF).cuda(), cache, dev(table), w.cuda(),
                                        dev([n], I32), topk, 1, 64, 4).cpu().numpy()[0, 0]
    assert np.array_equal(got, np.sort(np.argsort(-tiny, kind="stable")[:topk]))


def test_indexer_does_not_depend_on_the_batch():
    rng = np.random.default_rng(13)
    lens = [2000, 1500, 1999]
    cache, table, keys, q, w = index_case(rng, 3, 2, 64, 128, 4, lens, 4, 64, BF)
    whole = serve.csa_indexer_topk_decode(q.cuda(), cache, dev(table), w.cuda(), dev(lens, I32), 99, 4, 64, 4)
    for s in range(3):
        alone = serve.csa_indexer_topk_decode(q[s:s + 1].cuda(), cache, dev(table[s:s + 1]), w[s:s + 1].cuda(),
                                              dev(lens[s:s + 1], I32), 99, 4, 64, 4)
        assert torch.equal(alone[0], whole[s])


def test_indexer_long_row():
    """One row over many tiles and several thousand places, against fp64 torch."""
    rng = np.random.default_rng(14)
    for bits, n, topk in ((4, 70001, 1024), (8, 30000, 5000)):
        d, H, page = 128, 64, 64
        keys = torch.from_numpy(rng.standard_normal((1, n, d)).astype(np.float32)).to(BF)
        cache, table, keys, q, w = index_case(rng, 1, 1, H, d, 1, [n], bits, page, BF, keys=keys)
        held = torch.zeros(1, n, d, dtype=F32, device="cuda")
        serve.csa_cache_read(cache, dev(table), dev(np.zeros(1, np.int32)), held, page, bits)
        score = ((held[0].double() @ q[0, 0].cuda().double().T).clamp(min=0)
                 * w[0, 0].cuda().double()).sum(1)
        want = score.sort(descending=True, stable=True).indices[:topk].sort().values
        got = serve.csa_indexer_topk_decode(q.cuda(), cache, dev(table), w.cuda(), dev([n], I32), topk, 1,
                                            page, bits)
        assert torch.equal(got[0, 0].long(), want)


@pytest.mark.parametrize("n,kind", [(300000, "random"), (300000, "ties"), (40000, "ties"),
                                    (40000, "outlier")])
def test_indexer_rows_of_several_ctas(n, kind):
    """Rows beyond what one CTA, and beyond what eight, keep in shared memory;
    rows of ties, and rows whose range one outlier stretches."""
    rng = np.random.default_rng(n)
    d, H, page, bits, topk = 64, 8, 64, 8, 700
    keys = rng.standard_normal((1, n, d)).astype(np.float32)
    if kind == "ties":
        keys = keys[:, rng.integers(0, 3, n)]
    if kind == "outlier":
        keys[0, 777] *= 1e6
    keys = torch.from_numpy(keys).to(BF)
    cache, table, keys, q, w = index_case(rng, 1, 1, H, d, 1, [n], bits, page, BF, keys=keys)
    w = w.abs()
    held = torch.zeros(1, n, d, dtype=F32, device="cuda")
    serve.csa_cache_read(cache, dev(table), dev(np.zeros(1, np.int32)), held, page, bits)
    score = ((held[0].double() @ q[0, 0].cuda().double().T).clamp(min=0) * w[0, 0].cuda().double()).sum(1)
    want = score.sort(descending=True, stable=True).indices[:topk].sort().values
    got = serve.csa_indexer_topk_decode(q.cuda(), cache, dev(table), w.cuda(), dev([n], I32), topk, 1, page,
                                        bits)
    assert torch.equal(got[0, 0].long(), want)


@pytest.mark.parametrize("n,dtype,H,d", [(2000, BF, 16, 64), (40000, BF, 16, 64), (2000, F32, 4, 96),
                                         (700, BF, 64, 128)])
def test_indexer_rows_with_nan_and_infinite_inputs(n, dtype, H, d):
    """Such a row gets blocks of its own in ascending order; the others are exact."""
    b, page, topk = 6, 64, 300
    rng = np.random.default_rng(n + d)
    cache, table, keys, q, w = index_case(rng, b, 1, H, d, 1, [n] * b, 4, page, dtype)
    w[0, 0, H // 2] = float("nan")
    w[1, 0, 0] = float("inf")
    q[2, 0, 1, 5] = float("nan")
    q[3, 0] = float("inf")
    w[3, 0, :] = -1.0
    # keys that nothing has written: NaN codes and infinite scales
    cache[dev(table[4, 1:3]).long()] = POISON
    got = serve.csa_indexer_topk_decode(q.cuda(), cache, dev(table), w.cuda(), dev([n] * b, I32), topk, 1,
                                        page, 4).cpu().numpy()
    assert csa.csa_get_device_status() == 0
    for s in range(b):
        assert got[s, 0, 0] >= 0 and got[s, 0, -1] < n and (np.diff(got[s, 0]) > 0).all()
    want = orc.index_row(f64(q)[5, 0], f64(w)[5, 0], orc.held_rows(f64(keys[5]), 4), n - 1, 1, topk)
    assert np.array_equal(got[5, 0], want)


def test_indexer_bad_page_and_length():
    rng = np.random.default_rng(15)
    n, page = 200, 16
    cache, table, keys, q, w = index_case(rng, 2, 1, 16, 64, 1, [n, n], 4, page, BF)
    table = table.copy()
    table[1, 3] = cache.shape[0]                        # keys 48..63 of sequence 1 score as zero keys
    got = serve.csa_indexer_topk_decode(q.cuda(), cache, dev(table), w.cuda(), dev([n, n], I32), 30, 1, page,
                                        4).cpu().numpy()
    assert csa.csa_get_device_status(with_site=True) == (DEVICE_CHECK, SITE_PAGE)
    held = [orc.held_rows(f64(keys[s]), 4) for s in range(2)]
    held[1][48:64] = 0.0
    for s in range(2):
        assert np.array_equal(got[s, 0], orc.index_row(f64(q)[s, 0], f64(w)[s, 0], held[s], n - 1, 1, 30))
    # a length beyond the table is clamped to its slots, a negative one is empty
    got = serve.csa_indexer_topk_decode(q.cuda(), cache, dev(table * 0 + np.arange(13), I32), w.cuda(),
                                        dev([-5, 100000], I32), 208, 1, page, 4).cpu().numpy()
    assert csa.csa_get_device_status(with_site=True) == (DEVICE_CHECK, SITE_RANGE)
    assert (got[0] == -1).all() and np.array_equal(got[1, 0], np.arange(208))


# --------------------------------------------------------------- attention

def check_row(o, lse, q, raw, cmp, idx, sink, scale, t, ratio, window, dtype):
    """Bounds: a logit's fp32 dot errs by at most d 2^-23 of sum |q k| (products
    summed in fp32, every sum rounded once), and e^x - 1 ~ x.  bf16 attention
    may round each probability to bf16 (half a step: 2^-8 relative, with their
    sum 2^-8 more) and rounds o once (2^-8); fp32 rounds nothing to fewer bits."""
    want, want_lse, spread = orc.attend_row(q, raw, cmp, idx, sink, scale, t, ratio, window)
    d = q.shape[-1]
    big = 0.0
    if t >= 0:
        top = max(np.abs(raw(p)).max() for p in range(max(0, t - window + 1), t + 1))
        js = range((t + 1) // ratio) if idx is None else [j for j in idx if 0 <= j < (t + 1) // ratio]
        for j in js:
            top = max(top, np.abs(cmp(int(j))).max())
        big = np.abs(q).sum(-1).max() * top * scale
    logit = 2 * d * 2.0 ** -23 * big + 2.0 ** -20
    rel = logit + (2 * 2.0 ** -8 if dtype == BF else 0.0)
    tol = rel * spread + (2.0 ** -8 if dtype == BF else 2.0 ** -23) * np.abs(want) + 1e-30
    got = f64(o)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())
    got_lse = f64(lse)
    inf = np.isinf(want_lse)
    assert np.array_equal(got_lse[inf], want_lse[inf])
    assert (np.abs(got_lse[~inf] - want_lse[~inf]) <= logit + 2.0 ** -22 * np.abs(want_lse[~inf])).all()


ATTN_CASES = [
    # b, s_q, H, d, ratio, window, lens, K (0: idx None; -1: no compressed rows), bits, page, dtype, sink
    (1, 1, 32, 128, 4, 128, [700], 64, 4, 64, BF, True),
    (5, 1, 32, 128, 4, 31, [0, 1, 5, 300, 1029], 100, 8, 64, BF, True),
    (2, 3, 32, 128, 128, 128, [2, 1500], 0, 4, 64, BF, False),
    (2, 1, 64, 512, 4, 128, [900, 77], 130, 4, 16, BF, True),
    (2, 2, 64, 512, 4, 65, [515, 1], 33, 8, 48, BF, True),
    (3, 1, 16, 64, 4, 16, [200, 16, 64], 17, 4, 16, BF, False),
    (1, 2, 8, 64, 1, 7, [333], 0, 8, 16, BF, True),
    (2, 1, 64, 256, 4, 100, [401, 640], 50, 4, 64, BF, True),
    (1, 1, 3, 96, 2, 40, [150], 20, 8, 16, BF, False),
    (1, 1, 128, 128, 4, 64, [260], 300, 4, 16, BF, True),
    (2, 2, 32, 128, 4, 50, [90, 300], -1, 4, 16, BF, True),
    (2, 1, 64, 512, 1, 1, [600, 1], 0, 4, 64, BF, False),
    (2, 1, 8, 128, 4, 33, [500, 3], 40, 4, 16, F32, True),
    (1, 2, 5, 160, 4, 12, [320], 0, 8, 32, F32, False),
    (1, 1, 32, 512, 4, 128, [1000], 64, 4, 64, F32, True),
]


def attn_case(rng, case):
    b, s_q, H, d, ratio, window, lens, K, bits, page, dtype, with_sink = case
    n_c = max(1, max(lens) // ratio)
    P_raw = -(-(window + s_q - 1) // page)
    P_cmp = -(-n_c // page)
    n_pages, (raw_t, cmp_t) = tables(rng, b, P_raw, P_cmp)
    cache = empty_cache(n_pages, page, d, bits)
    raw = torch.from_numpy(rng.standard_normal((b, max(max(lens), 1), d))).to(BF)
    cmp = torch.from_numpy(rng.standard_normal((b, n_c, d))).to(BF)
    serve.csa_cache_write(raw.cuda(), cache, dev(raw_t), dev(np.zeros(b, np.int32)), page, bits,
                          counts=dev(lens, I32))
    serve.csa_cache_write(cmp.cuda(), cache, dev(cmp_t), dev(np.zeros(b, np.int32)), page, bits,
                          counts=dev([n // ratio for n in lens], I32))
    idx = None
    if K > 0:
        # repeats, -1 and entries that are not visible yet, in no order
        idx = rng.integers(-1, n_c + 3, (b, s_q, K)).astype(np.int32)
        idx[0, 0, :] = -1 if lens[0] > 200 else idx[0, 0]
        idx[-1, -1, K // 2:] = -1
    q = torch.from_numpy(rng.standard_normal((b, s_q, H, d))).to(dtype)
    sink = rng.standard_normal(H).astype(np.float32) if with_sink else None
    return cache, raw_t, (None if K < 0 else cmp_t), raw, cmp, idx, q, sink


def run_attn(case, parts, **kw):
    b, s_q, H, d, ratio, window, lens, K, bits, page, dtype, _ = case
    cache, raw_t, cmp_t, raw, cmp, idx, q, sink = parts
    return serve.csa_attn_decode(q.cuda(), cache, dev(raw_t), None if cmp_t is None else dev(cmp_t),
                                 None if idx is None else dev(idx), None if sink is None else dev(sink),
                                 dev(lens, I32), d ** -0.5, ratio, window, page, bits, **kw)


@pytest.mark.parametrize("case", ATTN_CASES, ids=lambda c: f"b{c[0]}s{c[1]}H{c[2]}d{c[3]}r{c[4]}K{c[7]}_{c[8]}bit")
def test_attention_matches_oracle(case):
    b, s_q, H, d, ratio, window, lens, K, bits, page, dtype, _ = case
    rng = np.random.default_rng(H + d + window)
    parts = attn_case(rng, case)
    cache, raw_t, cmp_t, raw, cmp, idx, q, sink = parts
    o, lse = run_attn(case, parts)
    assert o.dtype == dtype and o.shape == q.shape and lse.dtype == F32
    assert csa.csa_get_device_status() == 0
    for s in range(b):
        r = orc.held_rows(f64(raw[s, :max(1, lens[s])]), bits)
        c = orc.held_rows(f64(cmp[s]), bits)
        for i in range(s_q):
            rows = [] if K < 0 else None if idx is None else idx[s, i]
            check_row(o[s, i], lse[s, i], f64(q)[s, i], lambda p: r[p], lambda j: c[j], rows, sink,
                      d ** -0.5, lens[s] - s_q + i, ratio, window, dtype)


WIDE_CASES = [
    # 512 channels and 33 to 64 columns: heads of one query, of several, in groups of 64
    (2, 3, 16, 512, 4, 65, [515, 2], 0, 8, 16, BF, True),
    (1, 2, 32, 512, 128, 128, [1300], 0, 4, 64, BF, False),
    (2, 1, 96, 512, 4, 64, [300, 64], 40, 4, 16, BF, True),
    (1, 1, 33, 512, 2, 17, [90], 70, 8, 48, BF, False),
    (3, 2, 64, 512, 4, 200, [1, 0, 450], -1, 4, 64, BF, True),
    (1, 1, 128, 512, 4, 1, [5], 0, 8, 16, BF, False),
    (1, 5, 16, 512, 1, 3, [700], 0, 4, 32, BF, True),
]


@pytest.mark.parametrize("case", WIDE_CASES, ids=lambda c: f"b{c[0]}s{c[1]}H{c[2]}r{c[4]}K{c[7]}_{c[8]}bit")
def test_attention_at_512_channels(case):
    test_attention_matches_oracle(case)


@pytest.mark.parametrize("H,d,s_q,K,bits", [(64, 512, 1, 1000, 4), (64, 512, 1, 0, 8), (16, 512, 4, 0, 4),
                                             (32, 512, 1, 0, 4), (32, 128, 1, 1000, 8), (64, 256, 1, 0, 4)])
def test_attention_whose_maximum_keeps_growing(H, d, s_q, K, bits):
    """Rows along one direction, longer from slot to slot, up to logits of about
    200: every tile's maximum is above those before, and the last few slots
    have all the weight.  40 sequences: several tiles to a CTA."""
    b, n = 40, 4400
    case = (b, s_q, H, d, 4, 64, [n] * b, K, bits, 64, BF, True)
    rng = np.random.default_rng(H + d + s_q)
    n_pages, (raw_t, cmp_t) = tables(rng, b, 2, -(-(n // 4) // 64))
    cache = empty_cache(n_pages, 64, d, bits)
    u = np.sign(rng.standard_normal(d))
    ramp = np.linspace(0.01, 1.0, n // 4)[:, None]
    cmp = torch.from_numpy(ramp * u + 0.02 * rng.standard_normal((n // 4, d))).to(BF)[None]
    raw = torch.from_numpy(0.01 * rng.standard_normal((128, d))).to(BF)[None]     # of the last positions
    serve.csa_cache_write(raw.cuda().expand(b, -1, -1), cache, dev(raw_t), dev([n - 128] * b, I32), 64, bits)
    serve.csa_cache_write(cmp.cuda().expand(b, -1, -1), cache, dev(cmp_t), dev([0] * b, I32), 64, bits)
    idx = np.broadcast_to(np.arange(1100 - K, 1100, dtype=np.int32), (b, s_q, K)).copy() if K else None
    q = torch.from_numpy(200 * d ** -0.5 * u + rng.standard_normal((b, s_q, H, d))).to(BF)
    sink = rng.standard_normal(H).astype(np.float32)
    o, lse = run_attn(case, (cache, raw_t, cmp_t, raw, cmp, idx, q, sink))
    assert csa.csa_get_device_status() == 0
    r, c = orc.held_rows(f64(raw[0]), bits), orc.held_rows(f64(cmp[0]), bits)
    for s in (0, b - 1):
        for i in range(s_q):
            check_row(o[s, i], lse[s, i], f64(q[s, i]), lambda p: r[p - n + 128], lambda j: c[j],
                      None if idx is None else idx[s, i], sink, d ** -0.5, n - s_q + i, 4, 64, BF)


@pytest.mark.parametrize("H,d,bits", [(16, 128, 4), (16, 128, 8), (16, 512, 4), (16, 512, 8), (32, 64, 8),
                                      (8, 96, 8)])
def test_attention_rows_that_only_a_later_query_sees(H, d, bits):
    """The newest token's row has NaN, infinities and magnitudes at the end of
    fp32; the queries before it share its CTA, and do not see it."""
    case = (1, 3, H, d, 4, 40, [600], 0, bits, 16, BF, True)
    rng = np.random.default_rng(H + d + bits)
    cache, raw_t, cmp_t, raw, cmp, idx, q, sink = attn_case(rng, case)
    n = 600
    bad = torch.from_numpy(rng.standard_normal((1, 1, d))).float()
    bad[0, 0, ::3] = float("inf")
    bad[0, 0, 1::7] = float("nan")
    bad[0, 0, 2::5] = -3.4e38
    serve.csa_cache_write(bad.cuda(), cache, dev(raw_t), dev([n - 1], I32), 16, bits)
    got = torch.empty(1, 1, d, dtype=BF, device="cuda")
    serve.csa_cache_read(cache, dev(raw_t), dev([n - 1], I32), got, 16, bits)
    assert bool(torch.isfinite(got).all())
    o, lse = run_attn(case, (cache, raw_t, cmp_t, raw, cmp, idx, q, sink))
    r, c = orc.held_rows(f64(raw[0]), bits), orc.held_rows(f64(cmp[0]), bits)
    for i in range(2):
        check_row(o[0, i], lse[0, i], f64(q)[0, i], lambda p: r[p], lambda j: c[j], None, sink, d ** -0.5,
                  n - 3 + i, 4, 40, BF)


def test_attention_large_logits_and_dominant_sink():
    """Logits of several hundred: the running maximum carries them; a sink far
    above them leaves o near zero, far below it changes nothing."""
    case = (1, 1, 32, 128, 4, 64, [400], 80, 8, 16, BF, True)
    rng = np.random.default_rng(21)
    cache, raw_t, cmp_t, raw, cmp, idx, q, sink = attn_case(rng, case)
    q = q * 30
    r, c = orc.held_rows(f64(raw[0]), 8), orc.held_rows(f64(cmp[0]), 8)
    for level in (-1000.0, 1000.0):
        s = np.full(32, level, np.float32)
        o, lse = run_attn(case, (cache, raw_t, cmp_t, raw, cmp, idx, q, s))
        check_row(o[0, 0], lse[0, 0], f64(q)[0, 0], lambda p: r[p], lambda j: c[j], idx[0, 0], s, 128 ** -0.5,
                  399, 4, 64, BF)


def test_attention_bad_page_is_masked():
    case = (2, 1, 16, 64, 1, 16, [100, 100], 0, 4, 16, BF, True)
    rng = np.random.default_rng(22)
    parts = list(attn_case(rng, case))
    cache, raw_t, cmp_t, raw, cmp, idx, q, sink = parts
    cmp_t = cmp_t.copy()
    cmp_t[1, 2] = -7                                    # blocks 32..47 of sequence 1
    parts[2] = cmp_t
    o, lse = run_attn(case, parts)
    assert csa.csa_get_device_status(with_site=True) == (DEVICE_CHECK, SITE_PAGE)
    for s in range(2):
        r, c = orc.held_rows(f64(raw[s]), 4), orc.held_rows(f64(cmp[s]), 4)
        rows = [j for j in range(100) if s == 0 or not 32 <= j < 48]
        check_row(o[s, 0], lse[s, 0], f64(q)[s, 0], lambda p: r[p], lambda j: c[j], rows, sink, 0.125, 99, 1,
                  16, BF)


def test_attention_is_the_same_bits_every_time():
    case = (2, 1, 64, 512, 4, 128, [900, 1700], 300, 4, 64, BF, True)
    parts = attn_case(np.random.default_rng(23), case)
    o, lse = run_attn(case, parts)
    for _ in range(3):
        o2, lse2 = run_attn(case, parts)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


# ---------------------------------------------- streams, graphs, together

def test_allocations_of_a_call_on_a_given_stream_belong_to_it():
    """While the call waits behind other work of its stream, tensors of the sizes that
    it allocated are made and filled on the current one: they keep what they hold."""
    rng = np.random.default_rng(32)
    n, page, topk = 9000, 64, 100
    icache, itable, keys, qi, w = index_case(rng, 2, 1, 64, 128, 1, [n, n], 4, page, BF)
    case = (1, 1, 64, 128, 4, 64, [n], 0, 4, page, BF, True)
    cache, raw_t, cmp_t, raw, cmp, idx, q, sink = attn_case(rng, case)
    i_args = [qi.cuda(), icache, dev(itable), w.cuda(), dev([n, n], I32), topk, 1, page, 4]
    a_args = [q.cuda(), cache, dev(raw_t), dev(cmp_t), None, dev(sink), dev([n], I32), 128 ** -0.5, 4, 64, page, 4]
    want = [serve.csa_indexer_topk_decode(*i_args), *serve.csa_attn_decode(*a_args)]
    sizes = [serve.csa_indexer_topk_decode_workspace_size(2, 1, 64, 128, itable.shape[1] * page),
             serve.csa_attn_decode_workspace_size(1, 1, 64, 128, 64, cmp_t.shape[1] * page)]
    assert min(sizes) > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    got = [serve.csa_indexer_topk_decode(*i_args, stream=side), *serve.csa_attn_decode(*a_args, stream=side)]
    mine = [torch.full((max(k, 16),), 7, dtype=U8, device="cuda") for k in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool((m == 7).all()) for m in mine)
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_calls_on_a_side_stream_and_in_two_graphs_that_share_workspaces():
    rng = np.random.default_rng(31)
    case = (2, 1, 32, 128, 4, 64, [500, 300], 50, 4, 16, BF, True)
    parts = attn_case(rng, case)
    cache, raw_t, cmp_t, raw, cmp, idx, q, sink = parts
    icache, itable, keys, qi, w = index_case(rng, 2, 1, 64, 128, 4, [500, 300], 4, 16, BF)
    args = [dev(raw_t), dev(cmp_t), dev(sink), dev([500, 300], I32), dev(itable), qi.cuda(), w.cuda(), q.cuda()]
    rt, ct, sk, lens, it, qi_d, w_d, q_d = args
    ws_i = torch.empty(serve.csa_indexer_topk_decode_workspace_size(2, 1, 64, 128, it.shape[1] * 16), dtype=U8,
                       device="cuda")
    ws_a = torch.empty(serve.csa_attn_decode_workspace_size(2, 1, 32, 128, 64, 50), dtype=U8, device="cuda")

    def step(out_idx, o, lse):
        serve.csa_indexer_topk_decode(qi_d, icache, it, w_d, lens, 50, 4, 16, 4, workspace=ws_i, out_idx=out_idx)
        serve.csa_attn_decode(q_d, cache, rt, ct, out_idx, sk, lens, 128 ** -0.5, 4, 64, 16, 4, workspace=ws_a,
                              out=o, lse=lse)

    def bufs():
        return (torch.zeros(2, 1, 50, dtype=I32, device="cuda"), torch.zeros_like(q_d),
                torch.zeros(2, 1, 32, device="cuda"))

    ref = bufs()
    step(*ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bufs()
    with torch.cuda.stream(side):
        step(*got)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, got))

    graphs = []
    for _ in range(2):
        out = bufs()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(*out)
        graphs.append((g, out))
    for (g, out) in graphs:
        for t in out:
            t.zero_()
        g.replay()
        g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(x, y) for x, y in zip(ref, out))
    # a replay reads the buffers as they are then: shorter sequences
    lens.copy_(dev([77, 12], I32))
    want = bufs()
    step(*want)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, graphs[0][1]))
    assert not torch.equal(want[1], ref[1])


def test_two_calls_at_once_on_two_streams():
    rng = np.random.default_rng(33)
    case = (3, 1, 64, 512, 4, 128, [900, 5, 1300], 200, 4, 16, BF, True)
    parts = attn_case(rng, case)
    icache, itable, keys, qi, w = index_case(rng, 3, 1, 64, 128, 4, [40000, 9000, 100], 4, 64, BF)
    lens = dev([40000, 9000, 100], I32)
    qi, w, itable = qi.cuda(), w.cuda(), dev(itable)
    want_o, want_l = run_attn(case, parts)
    want_i = serve.csa_indexer_topk_decode(qi, icache, itable, w, lens, 512, 4, 64, 4)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for r in range(6):
        with torch.cuda.stream(streams[r % 2]):
            got.append((run_attn(case, parts),
                        serve.csa_indexer_topk_decode(qi, icache, itable, w, lens, 512, 4, 64, 4)))
    torch.cuda.synchronize()
    for (o, lse), idx in got:
        assert torch.equal(o, want_o) and torch.equal(lse, want_l) and torch.equal(idx, want_i)


def test_many_short_sequences():
    """More queries than a grid dimension of 65535 CTAs times two head groups."""
    b, H, d, page, bits = 33000, 128, 64, 16, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = empty_cache(3, page, d, bits)
    table = torch.ones(b, 1, dtype=I32, device="cuda")
    raw = torch.randn(1, 4, d, generator=g, device="cuda").to(BF)
    serve.csa_cache_write(raw, cache, table[:1], torch.zeros(1, dtype=I32, device="cuda"), page, bits)
    q = torch.randn(b, 1, H, d, generator=g, device="cuda").to(BF)
    lens = (torch.arange(b, device="cuda") % 5).to(I32)
    o, lse = serve.csa_attn_decode(q, cache, table, None, None, None, lens, 0.125, 4, 3, page, bits)
    held = torch.zeros(1, 4, d, dtype=F32, device="cuda")
    serve.csa_cache_read(cache, table[:1], torch.zeros(1, dtype=I32, device="cuda"), held, page, bits)
    z = (q[:, 0].double() @ held[0].double().T) * 0.125
    pos = torch.arange(4, device="cuda")
    t = lens.long()[:, None] - 1
    ok = (pos <= t) & (pos > t - 3)
    z = torch.where(ok[:, None], z, torch.full_like(z, -float("inf")))
    want = torch.softmax(z, -1).nan_to_num(0.0) @ held[0].double()
    # probabilities, their sum and o in bf16 half steps, as in check_row
    spread = torch.softmax(z, -1).nan_to_num(0.0) @ held[0].double().abs()
    assert bool(((o[:, 0].double() - want).abs() <= 3 * 2.0 ** -8 * spread + 1e-4).all())
    assert bool((lse[lens == 0] == -float("inf")).all())


FUZZ = list(range(24))


@pytest.mark.parametrize("seed", FUZZ)
def test_random_configurations(seed):
    """A random layer: cache rows written in ragged pieces over a ring, selected
    and attended to, against fp64 torch on the rows read back."""
    import random
    r = random.Random(seed)
    rng = np.random.default_rng(seed)
    b, s_q, bits = r.randint(1, 6), r.choice([1, 1, 2, 3, 5]), r.choice([4, 8])
    page, ratio = r.choice([16, 32, 48, 64]), r.choice([1, 2, 4, 16])
    H, d = r.choice([1, 8, 16, 24, 32, 64, 96]), r.choice([32, 64, 128, 192, 256, 512])
    H_I, d_I, topk = r.choice([1, 4, 16, 40, 64, 128]), r.choice([32, 64, 128, 256]), r.choice([1, 9, 64, 257])
    window = r.choice([1, 5, 40, 128])
    dtype = r.choice([BF, BF, BF, F32])
    lens = [r.choice([0, 1, r.randint(2, 60), r.randint(60, 1500)]) for _ in range(b)]
    n_c = max(1, max(lens) // ratio)
    P_raw, P_cmp = -(-(window + s_q - 1) // page) + r.randint(0, 2), -(-n_c // page)
    n_pages, (raw_t, cmp_t) = tables(rng, b, P_raw, P_cmp)
    i_pages, (key_t,) = tables(rng, b, P_cmp)
    raw_t, cmp_t, key_t, seq = dev(raw_t), dev(cmp_t), dev(key_t), dev(lens, I32)
    cache, icache = empty_cache(n_pages, page, d, bits), empty_cache(i_pages, page, d_I, bits)
    top = max(max(lens), 1)
    raw = torch.from_numpy(rng.standard_normal((b, top, d))).to(dtype).cuda()
    cmp = torch.from_numpy(rng.standard_normal((b, n_c, d))).to(dtype).cuda()
    keys = torch.from_numpy(rng.standard_normal((b, n_c, d_I))).to(dtype).cuda()
    zero = torch.zeros(b, dtype=I32, device="cuda")
    cut = top // 3
    first = torch.minimum(seq, torch.full_like(seq, cut))
    serve.csa_cache_write(raw[:, :max(cut, 1)], cache, raw_t, zero, page, bits, counts=first)
    serve.csa_cache_write(raw[:, cut:], cache, raw_t, first, page, bits, counts=seq - first)
    serve.csa_cache_write(cmp, cache, cmp_t, zero, page, bits, counts=seq // ratio)
    serve.csa_cache_write(keys, icache, key_t, zero, page, bits, counts=seq // ratio)
    q = torch.from_numpy(rng.standard_normal((b, s_q, H, d))).to(dtype).cuda()
    q_I = torch.from_numpy(rng.standard_normal((b, s_q, H_I, d_I))).to(dtype).cuda()
    w = torch.from_numpy(rng.standard_normal((b, s_q, H_I))).float().cuda()
    sink = torch.from_numpy(rng.standard_normal(H)).float().cuda() if r.random() < 0.7 else None
    idx = serve.csa_indexer_topk_decode(q_I, icache, key_t, w, seq, topk, ratio, page, bits)
    use = None if r.random() < 0.3 else idx
    o, lse = serve.csa_attn_decode(q, cache, raw_t, cmp_t, use, sink, seq, d ** -0.5, ratio, window, page, bits)
    assert csa.csa_get_device_status() == 0
    k_held = serve.csa_cache_read(icache, key_t, zero, torch.zeros(b, n_c, d_I, device="cuda"), page, bits,
                                  counts=seq // ratio)
    c_held = serve.csa_cache_read(cache, cmp_t, zero, torch.zeros(b, n_c, d, device="cuda"), page, bits,
                                  counts=seq // ratio)
    keep = min(P_raw * page, window + s_q - 1)
    start = (seq - keep).clamp(min=0)
    r_held = serve.csa_cache_read(cache, raw_t, start, torch.zeros(b, keep, d, device="cuda"), page, bits,
                                  counts=seq - start)
    for s in range(b):
        for i in range(s_q):
            t = lens[s] - s_q + i
            vis = (t + 1) // ratio if t >= 0 else 0
            sc = ((k_held[s, :vis].double() @ q_I[s, i].double().T).clamp(min=0) * w[s, i].double()).sum(1)
            want = sc.sort(descending=True, stable=True).indices[:topk].sort().values
            got = idx[s, i]
            assert torch.equal(got[:len(want)].long(), want) and bool((got[len(want):] == -1).all()), (s, i)
            rows = torch.zeros(0, d, dtype=torch.float64, device="cuda")
            if t >= 0:
                p0 = max(0, t - window + 1)
                off = int(start[s])
                js = idx[s, i][idx[s, i] >= 0].long() if use is not None else torch.arange(vis, device="cuda")
                rows = torch.cat([r_held[s, p0 - off:t + 1 - off], c_held[s][js]]).double()
            z = q[s, i].double() @ rows.T * d ** -0.5
            zs = sink.double()[:, None] if sink is not None else torch.full((H, 1), -float("inf"), device="cuda",
                                                                        dtype=torch.float64)
            l = torch.logsumexp(torch.cat([z, zs], 1), 1)
            p = torch.exp(z - l[:, None])
            p = torch.where(torch.isfinite(p), p, torch.zeros_like(p))
            ref, spread = p @ rows, p @ rows.abs()
            # as in check_row: fp32 logits, probabilities and o in bf16 half steps
            big = (q[s, i].double().abs().sum(-1).max() * rows.abs().max() * d ** -0.5).item() if len(rows) else 0.0
            logit = 2 * d * 2.0 ** -23 * big + 2.0 ** -20
            tol = (logit + (2 * 2.0 ** -8 if dtype == BF else 0)) * spread + (
                2.0 ** -8 if dtype == BF else 2.0 ** -23) * ref.abs() + 1e-30
            assert bool(((o[s, i].double() - ref).abs() <= tol).all()), (s, i)
            fin = torch.isfinite(l)
            assert torch.equal(lse[s, i][~fin].double(), l[~fin])
            assert bool(((lse[s, i].double() - l)[fin].abs() <= logit + 2.0 ** -22 * l[fin].abs()).all())


@pytest.mark.parametrize("bits", [4, 8])
def test_decode_loop_matches_the_whole_sequence_calls(bits):
    """Token by token: append the raw row; at the end of a block pool it
    (csa_compress) and append the pooled row and the block's index key; select;
    attend.  The whole-sequence calls on the rows read back select the same
    blocks and give the same output up to both sides' rounding."""
    g = torch.Generator().manual_seed(41)
    b, n, H, d, H_I, d_I, ratio, window, topk, page = 2, 75, 32, 128, 64, 128, 4, 20, 6, 16
    kv = torch.randn(b, n, d, generator=g).to(BF).cuda()
    score = (torch.randn(b, n, d, generator=g) * 0.5).to(BF).cuda()
    keys = torch.randn(b, n // ratio, d_I, generator=g).to(BF).cuda()
    q = torch.randn(b, n, H, d, generator=g).to(BF).cuda()
    q_I = torch.randn(b, n, H_I, d_I, generator=g).to(BF).cuda()
    w = (torch.randn(b, n, H_I, generator=g) / 2).cuda()
    sink = torch.randn(H, generator=g).cuda()
    n_c = n // ratio
    rng = np.random.default_rng(42)
    P_all, P_cmp = -(-n // page), -(-n_c // page)
    n_pages, (raw_t, cmp_t) = tables(rng, b, P_all, P_cmp)
    i_pages, (key_t,) = tables(rng, b, P_cmp)
    raw_t, cmp_t, key_t = dev(raw_t), dev(cmp_t), dev(key_t)
    cache, icache = empty_cache(n_pages, page, d, bits), empty_cache(i_pages, page, d_I, bits)
    O = torch.zeros(b, n, H, d, dtype=BF, device="cuda")
    L = torch.zeros(b, n, H, device="cuda")
    idx = torch.full((b, n, topk), -1, dtype=I32, device="cuda")
    for t in range(n):
        at = torch.full((b,), t, dtype=I32, device="cuda")
        serve.csa_cache_write(kv[:, t:t + 1], cache, raw_t, at, page, bits)
        if (t + 1) % ratio == 0:
            blk = (t + 1) // ratio - 1
            jj = torch.full((b,), blk, dtype=I32, device="cuda")
            pooled = csa.csa_compress(kv[:, t + 1 - ratio:t + 1].contiguous(),
                                      score[:, t + 1 - ratio:t + 1].contiguous(), ratio)
            serve.csa_cache_write(pooled, cache, cmp_t, jj, page, bits)
            serve.csa_cache_write(keys[:, blk:blk + 1], icache, key_t, jj, page, bits)
        lens = at + 1
        idx[:, t:t + 1] = serve.csa_indexer_topk_decode(q_I[:, t:t + 1].contiguous(), icache, key_t,
                                                        w[:, t:t + 1].contiguous(), lens, topk, ratio, page, bits)
        o, l = serve.csa_attn_decode(q[:, t:t + 1].contiguous(), cache, raw_t, cmp_t,
                                     idx[:, t:t + 1].contiguous(), sink, lens, d ** -0.5, ratio, window, page,
                                     bits)
        O[:, t:t + 1], L[:, t:t + 1] = o, l
    zero = torch.zeros(b, dtype=I32, device="cuda")
    kv_full = torch.empty(b, n + n_c, d, dtype=BF, device="cuda")
    serve.csa_cache_read(cache, raw_t, zero, kv_full[:, :n], page, bits)
    serve.csa_cache_read(cache, cmp_t, zero, kv_full[:, n:], page, bits)
    k_I = serve.csa_cache_read(icache, key_t, zero, torch.empty(b, n_c, d_I, dtype=BF, device="cuda"), page, bits)
    ref_idx = csa.csa_indexer_topk(q_I, k_I, w, topk, ratio)
    assert torch.equal(idx[..., :ref_idx.shape[2]], ref_idx)
    ref_o, ref_l = csa.csa_attn_fwd(q, kv_full, idx, sink, d ** -0.5, ratio, window)
    # each side: probabilities and their sum rounded to bf16 (2 x 2^-8) and o rounded once (2^-8), of at
    # most the largest |v| of the row's slots
    top = kv_full.float().abs().max().item()
    assert (O.float() - ref_o.float()).abs().max().item() <= 2 * 3 * 2.0 ** -8 * top
    rel = (O.float() - ref_o.float()).norm() / ref_o.float().norm()
    assert rel.item() <= 2 * 3 * 2.0 ** -8
    assert (L - ref_l).abs().max().item() <= 1e-4
    assert csa.csa_get_device_status() == 0
