"""Numerics of the serving calls where an ordinary input does not reach them, on
the GPU against the fp64 oracle or against values known by construction."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_sum_gb300 import csa, serve
from oracle import serve_oracle as orc
from test_gpu_serve import BF, F32, attn_case, check_row, dev, empty_cache, f64, run_attn, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from compressed_sparse_attention_sum_gb300 import build
    build.build()
    serve.load_library()
    csa.csa_get_device_status()
    yield
    assert csa.csa_get_device_status() == 0


# --------------------------------------------------------------- attention

# b, s_q, H, d, K (0: every visible block), bits, dtype: one CTA a query, clusters, parts
# that a second kernel joins, several queries a CTA, CUDA cores
EVEN_CASES = [
    (1, 1, 32, 128, 600, 4, BF), (96, 1, 32, 128, 600, 8, BF), (2, 2, 16, 64, 0, 8, BF),
    (1, 1, 32, 128, 0, 4, BF), (130, 1, 64, 256, 300, 4, BF), (2, 1, 8, 512, 300, 8, BF),
    (130, 1, 64, 512, 300, 4, BF), (3, 1, 64, 512, 700, 8, BF), (2, 3, 16, 512, 0, 4, BF),
    (80, 2, 64, 64, 0, 4, BF), (1, 1, 5, 96, 100, 4, BF), (2, 1, 16, 128, 200, 8, F32),
]


@pytest.mark.parametrize("case", EVEN_CASES, ids=lambda c: f"b{c[0]}s{c[1]}H{c[2]}d{c[3]}K{c[4]}_{c[5]}bit")
def test_attention_weights_add_up_to_one(case):
    """A channel that is 1 in every row comes out as exactly 1 (no sink), whatever the
    weights.  Fifteen rows of sixteen have the probability 2^-1 (1 + 2^-8 - 2^-12)
    relative to the others: rounded to bf16 it loses 2^-8 of itself, one step of the
    output, which every row shares unless the weights are divided by their own sum.
    What is left is fp32: with n = 64 to 2000 rows the sums err by less than
    n 2^-23 < 2^-12 of themselves, an eighth of half the bf16 step below 1 (2^-9)."""
    b, s_q, H, d, K, bits, dtype = case
    page, window, n = 16, 50, 2000
    rng = np.random.default_rng(d + H)
    n_pages, (raw_t, cmp_t) = tables(rng, b, -(-(window + s_q - 1) // page), -(-n // page))
    raw_t, cmp_t = dev(raw_t), dev(cmp_t)
    cache = empty_cache(n_pages, page, d, bits)
    rows = torch.zeros(b, n, d, device="cuda")
    rows[..., 0] = 1.0                                  # the constant channel
    rows[..., 33] = 1.0                                 # the one that q meets
    rows[:, ::16, 33] = 2.0
    zero = torch.zeros(b, dtype=torch.int32, device="cuda")
    lens = torch.full_like(zero, n)
    serve.csa_cache_write(rows, cache, raw_t, zero, page, bits)
    serve.csa_cache_write(rows, cache, cmp_t, zero, page, bits)
    p = 0.5 * (1 + 2.0 ** -8 - 2.0 ** -12)
    q = torch.zeros(b, s_q, H, d, dtype=dtype, device="cuda")
    q[..., 33] = 1.0
    idx = None
    if K:
        idx = dev(np.stack([np.sort(rng.permutation(n - s_q)[:K]) for _ in range(b * s_q)]).reshape(b, s_q, K),
                  torch.int32)
    o, lse = serve.csa_attn_decode(q, cache, raw_t, cmp_t, idx, None, lens, -float(np.log(p)), 1, window, page,
                                   bits)
    assert csa.csa_get_device_status() == 0
    # fp32 outputs keep what a bf16 one rounds away: the two sums of at most K + window terms (K > 0
    # here), each addition rounded by 2^-24 of them, (K + window) 2^-23 together, and a few more roundings
    # where parts are joined and divided
    off = (o[..., 0].double() - 1.0).abs().max().item()
    assert off <= ((K + window + 8) * 2.0 ** -23 if dtype == F32 else 0.0), off
    # the log of the weights' sum as they are, not as rounded: 2 -> e^(2 s), 1 -> e^s
    pos = torch.arange(n, device="cuda")
    for i in range(s_q):
        t = n - s_q + i
        js = pos[:t + 1].expand(b, -1) if idx is None else idx[:, i].long()
        twos = (js % 16 == 0).sum(1) + int((pos[t - window + 1:t + 1] % 16 == 0).sum())
        total = js.shape[1] + window
        s = -np.log(p)
        want = torch.log(twos.double() * np.exp(2 * s) + (total - twos).double() * np.exp(s))
        # logits are exact up to fp32 roundings of scale and of scale * log2 e (2^-23 of 2 s < 1.4), the
        # sum as above and one rounding of lse
        assert bool(((lse[:, i].double() - want[:, None]).abs() <= 2.0 ** -11).all())


# b, s_q, H, d, K (0: every visible block), bits, dtype
SINK_CASES = [(2, 1, 32, 128, 200, 4, BF), (100, 1, 16, 128, 40, 8, BF), (2, 3, 16, 128, 0, 4, BF), (1, 2, 32, 128, 0, 8, BF),
              (2, 1, 64, 512, 100, 4, BF), (100, 1, 64, 512, 40, 8, BF), (2, 2, 8, 512, 0, 4, BF), (2, 1, 5, 96, 60, 8, BF),
              (130, 1, 16, 64, 20, 4, F32), (2, 2, 16, 128, 300, 4, F32)]


@pytest.mark.parametrize("case", SINK_CASES, ids=lambda c: f"b{c[0]}s{c[1]}H{c[2]}d{c[3]}K{c[4]}_{c[5]}bit")
def test_attention_sinks_at_the_ends_of_fp32_and_empty_queries(case):
    """lse is the sink itself, to the bit, where a query has no row, and where the rows have no
    part in the denominator; a sink of fp32's lowest value or -inf changes nothing."""
    b, s_q, H, d, K, bits, dtype = case
    n = 700
    lens = [n] + [0] * (b - 1)
    spec = (b, s_q, H, d, 1, 33, lens, K, bits, 16, dtype, True)
    cache, raw_t, cmp_t, raw, cmp, idx, q, sink = attn_case(np.random.default_rng(H + d), spec)
    top = np.finfo(np.float32).max
    sink[:5] = [top, -top, -np.inf, 3e38, -2.5e38][:H]
    if idx is not None:
        idx[0] = np.arange(K)
    o, lse = run_attn(spec, (cache, raw_t, cmp_t, raw, cmp, idx, q, sink))
    assert csa.csa_get_device_status() == 0
    want = torch.from_numpy(sink).cuda()
    assert bool((o[1:] == 0).all()) and torch.equal(lse[1:], want.expand(b - 1, s_q, H))
    for h in (0, 3):
        assert bool((o[0, :, h] == 0).all()) and bool((lse[0, :, h] == want[h]).all())
    # the others, and heads without a weight for the sink, against the oracle
    r, c = orc.held_rows(f64(raw[0, :n]), bits), orc.held_rows(f64(cmp[0]), bits)
    rest = [h for h in range(H) if h not in (0, 3)]
    for i in range(s_q):
        t = n - s_q + i
        check_row(o[0, i, rest], lse[0, i, rest], f64(q)[0, i, rest], lambda p: r[p], lambda j: c[j],
                  None if idx is None else idx[0, i], sink[rest], d ** -0.5, t, 1, 33, dtype)


def test_attention_workspace_of_the_stated_bound_serves_every_batch():
    """One buffer of the bound for batches of 64 to 1 sequences, with results as with a workspace of
    the call's own; a buffer of the larger batch's size is refused by a smaller one."""
    d, H, page, n, K = 128, 32, 64, 3000, 512
    rng = np.random.default_rng(3)
    n_pages, (raw_t, cmp_t) = tables(rng, 64, 2, -(-n // page))
    raw_t, cmp_t = dev(raw_t), dev(cmp_t)
    cache = empty_cache(n_pages, page, d, 4)
    zero = torch.zeros(64, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn(64, n, d, generator=g, device="cuda").to(BF)
    serve.csa_cache_write(rows, cache, raw_t, zero, page, 4)
    serve.csa_cache_write(rows, cache, cmp_t, zero, page, 4)
    bound = torch.empty(2880 * (4 * d + 8) + 16, dtype=torch.uint8, device="cuda")
    for dtype in (BF, F32):
        for b in (64, 8, 1):
            q = torch.randn(b, 1, H, d, generator=g, device="cuda").to(dtype)
            idx = torch.randint(0, n, (b, 1, K), generator=g, device="cuda", dtype=torch.int32)
            for ix in (idx, None):
                args = (q, cache, raw_t[:b], cmp_t[:b], ix, None, zero[:b] + n, d ** -0.5, 1, 100, page, 4)
                want = serve.csa_attn_decode(*args)
                got = serve.csa_attn_decode(*args, workspace=bound)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    small = serve.csa_attn_decode_workspace_size(64, 1, H, d, 100, K)
    assert small < serve.csa_attn_decode_workspace_size(1, 1, H, d, 100, K)
    with pytest.raises(serve.CSAError):
        serve.csa_attn_decode(q, cache, raw_t[:1], cmp_t[:1], idx, None, zero[:1] + n, d ** -0.5, 1, 100, page, 4,
                              workspace=bound[:max(small, 16)])


# ----------------------------------------------------------------- indexer

def select(keys, q, w, topk, bits, page=64, dtype=BF):
    """Indices of one row: keys [n, d], q [H, d], w [H] (ratio 1, every key visible), and the
    oracle's on the rows held."""
    n, d = keys.shape
    P = -(-n // page)
    cache = empty_cache(P, page, d, bits)
    table = torch.arange(P, dtype=torch.int32, device="cuda")[None]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    serve.csa_cache_write(dev(keys, F32)[None].contiguous(), cache, table, zero, page, bits)
    q = dev(q, dtype)[None, None].contiguous()
    w = dev(w, F32)[None, None].contiguous()
    got = serve.csa_indexer_topk_decode(q, cache, table, w, dev([n], torch.int32), topk, 1, page, bits)
    held = serve.csa_cache_read(cache, table, zero, torch.zeros(1, n, d, device="cuda"), page, bits)
    assert np.array_equal(f64(held)[0], keys), "the keys are meant to be held exactly"
    assert csa.csa_get_device_status() == 0
    return got.cpu().numpy()[0, 0], orc.index_row(f64(q)[0, 0], f64(w)[0, 0], keys, n - 1, 1, topk)


@pytest.mark.parametrize("H", [1, 3, 16])
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, BF), (128, F32), (96, F32)])
def test_indexer_small_products_next_to_a_large_one(H, d, dtype):
    """Half of the blocks score 1 + (d - 2) 1.99 2^-26, in products of which a sum aligned to
    the large one keeps nothing; the others 1 + x, x just below that: what fp32 says is
    the wrong half, by nearly as much as a dot product can lose."""
    n, u = 200, 2.0 ** -24
    tail = 255 / 128 * 2.0 ** -26 * (d - 2)
    x = np.floor(tail / u / 8 * 0.95) * 8 * u               # 56 u at d = 128
    keys = np.zeros((n, d))
    keys[:, 0] = 1.0
    keys[0::2, 1] = 2.0 ** -6
    keys[1::2, 2:] = 2.0 ** -13
    q = np.zeros((H, d))
    q[0, 0], q[0, 1], q[0, 2:] = 1.0, x * 2.0 ** 6, 255 / 128 * 2.0 ** -13
    got, want = select(keys, q, np.ones(H), n // 2, 8, dtype=dtype)
    assert np.array_equal(want, np.arange(1, n, 2)) and x < tail
    assert np.array_equal(got, want)


def fp32_sets(keys, q, w, topk):
    """What fp32 scores alone would choose: the products added one by one, and 16 at a time
    (each step's exact sum added and rounded once)."""
    n, d = keys.shape
    k32, q32 = keys.astype(np.float32), q.astype(np.float32)
    one, step = np.zeros((n, len(q)), np.float32), np.zeros((n, len(q)), np.float32)
    for c in range(d):
        one = (one.astype(np.float64) + k32[:, c:c + 1].astype(np.float64) * q32[:, c]).astype(np.float32)
    for c in range(0, d, 16):
        step = (step + keys[:, c:c + 16] @ q[:, c:c + 16].T).astype(np.float32)
    out = []
    for dots in (one, step):
        score = np.zeros(n, np.float32)
        for h in range(len(q)):
            score = score + np.maximum(dots[:, h], 0) * np.float32(w[h])
        out.append(np.sort(np.argsort(-score, kind="stable")[:topk]))
    return out


def cancelling(rng, n, n_close, n_high, H):
    """Rows [n, 128] and q, w: of n_close blocks a product of 6 2^14 comes first and leaves last,
    and what decides between them, at most 6 2^-12, stands between; n_high blocks are far above,
    the others at zero."""
    keys = np.zeros((n, 128))
    kind = np.zeros(n, int)
    kind[rng.permutation(n)[:n_close + n_high]] = [1] * n_close + [2] * n_high
    live = kind > 0
    keys[live, 0], keys[live, 96], keys[live, 32] = 6.0, -6.0, 6.0
    keys[live, 33] = rng.choice([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], live.sum())
    keys[kind == 2, 64] = 6.0
    q = np.zeros((H, 128))
    q[:, 0], q[:, 96], q[:, 32], q[:, 33], q[:, 64] = 2.0 ** 14, 2.0 ** 14, 1.0, 2.0 ** -12, 4.0
    w = (np.abs(rng.standard_normal(H)) + 0.1).astype(np.float32).astype(np.float64)
    return keys, q, w


CLOSE_CASES = [
    # n, close blocks, blocks above, topk: one CTA; eight warps a block and several rounds; a row of several
    # CTAs; more close blocks than are ranked directly, in one CTA and in several
    (300, 300, 0, 40), (1000, 200, 30, 131), (20000, 300, 50, 170), (2000, 2000, 0, 333), (20000, 3000, 100, 900),
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype,H", [(BF, 32), (BF, 7), (F32, 8)])
@pytest.mark.parametrize("case", CLOSE_CASES, ids=lambda c: f"n{c[0]}close{c[1]}")
def test_indexer_close_blocks_are_chosen_by_their_exact_scores(case, dtype, H, bits):
    n, n_close, n_high, topk = case
    keys, q, w = cancelling(np.random.default_rng(n + H), n, n_close, n_high, H)
    got, want = select(keys, q, w, topk, bits, dtype=dtype)
    for wrong in fp32_sets(keys, q, w, topk):
        assert not np.array_equal(wrong, want)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype,H", [(BF, 64), (F32, 5)])
@pytest.mark.parametrize("n,topk", [(300, 101), (700, 211), (20000, 400)])
def test_indexer_exact_ties_whose_fp32_scores_differ(n, topk, dtype, H, bits):
    """All blocks score the same: their channels c and c + 64, at which q has equal values, are
    exchanged at random, so that fp32 sums see them in another order.  (The products are
    multiples of 2^-31 up to 2^5, which pairs of fp32 add without an error.)"""
    rng = np.random.default_rng(n + H)
    base = rng.choice([-6.0, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6], (64, 2))
    flip = rng.random((n, 64)) < 0.5
    keys = np.where(flip[..., None], base[None, :, ::-1], base[None]).transpose(0, 2, 1).reshape(n, 128)
    q = f64(torch.from_numpy(rng.standard_normal((H, 64))).bfloat16()) * 2.0 ** -rng.integers(0, 13, (H, 64))
    q = np.tile(q, 2)
    w = (np.abs(rng.standard_normal(H)) + 0.1).astype(np.float32).astype(np.float64)
    got, _ = select(keys, q, w, topk, bits, dtype=dtype)
    for wrong in fp32_sets(keys, q, w, topk):
        assert not np.array_equal(wrong, np.arange(topk))
    assert np.array_equal(got, np.arange(topk))


@pytest.mark.parametrize("dtype,H", [(BF, 32), (F32, 8)])
@pytest.mark.parametrize("q_e,w_e,k_e", [(-70, 0, 0), (-90, 0, 0), (-110, 0, 0), (-90, 90, 0), (60, 0, 0), (85, 0, 0),
                                         (85, -100, 0), (0, -110, 0), (0, -130, 0), (-60, 0, -60), (-100, 100, 30),
                                         (20, 0, 50), (-60, 100, -80)])
def test_indexer_is_exact_for_small_and_large_magnitudes(q_e, w_e, k_e, dtype, H):
    """The same rows with q, w and the keys times powers of two: the choice is the same, though
    squares of q, or products of w and q, leave fp32."""
    n, n_close, n_high, topk = 600, 300, 40, 130
    keys, q, w = cancelling(np.random.default_rng(H), n, n_close, n_high, H)
    keys, q = np.ldexp(keys, k_e), np.ldexp(q, q_e)
    w = np.ldexp(w, w_e).astype(np.float32).astype(np.float64)      # exponents below -126: rounded
    got, want = select(keys, q, w, topk, 4, dtype=dtype)
    assert np.array_equal(got, want)


# --------------------------------------------------- blocks as they complete

@pytest.mark.parametrize("ratio", [4, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_overlapping_blocks_pooled_as_they_complete(ratio, dtype):
    """csa_compress_overlap of the last two blocks: its second entry is the sequence's.  Both pool
    the same tokens in fp32 and cast once; the order of at most 256 terms may differ (2^-16 of
    sum w |kv| each way), which may move a cast by one step (2^-8, 2^-24 in fp32)."""
    g = torch.Generator(device="cuda").manual_seed(ratio)
    b, n, d = 2, 5 * ratio, 128
    kv = torch.randn(b, n, d, generator=g, device="cuda").to(dtype)
    score = torch.randn(b, n, d, generator=g, device="cuda").to(dtype)
    whole = csa.csa_compress_overlap(kv, score, ratio, 2)
    top = kv.abs().max().item()
    for j in range(1, n // ratio):
        last = slice((j - 1) * ratio, (j + 1) * ratio)
        got = csa.csa_compress_overlap(kv[:, last].contiguous(), score[:, last].contiguous(), ratio, 2)[:, 1]
        tol = 2.0 ** -15 * top + (2.0 ** -7 * top if dtype == BF else 0.0)
        assert (got.float() - whole[:, j].float()).abs().max().item() <= tol
