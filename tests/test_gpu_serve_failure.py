"""Waits of the serving calls that run out, without a fault: the test hook
csa_debug_arm_fault makes one CTA issue no product, so that its bounded waits (about
one second) give up with none in flight.  The call returns, also where that CTA
belongs to a cluster or writes one of several parts, the status word names the site,
nothing is written outside the outputs, and the next call is correct."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_sum_gb300 import csa, serve
from test_gpu_serve import BF, attn_case, dev, index_case, run_attn

pytestmark = pytest.mark.gpu

CSA_ERR_TIMEOUT, SITE_ATTN, SITE_INDEX = 5, 0x73, 0x74


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from compressed_sparse_attention_sum_gb300 import build
    build.build()
    serve.load_library()
    csa.csa_get_device_status()
    yield
    csa.csa_debug_arm_fault(0)
    assert csa.csa_get_device_status() == 0


def with_armed(site, call):
    csa.csa_debug_arm_fault(site)
    try:
        call()
        return csa.csa_get_device_status(with_site=True)
    finally:
        csa.csa_debug_arm_fault(0)


# b, s_q, H, d, ratio, window, lens, K, bits, page, dtype, sink
CASES = {
    "one CTA a query": (100, 1, 16, 128, 4, 64, [500] * 100, 40, 4, 16, BF, True),
    "a cluster": (1, 1, 32, 128, 4, 128, [3000], 500, 8, 64, BF, True),
    "clusters and a second kernel": (1, 2, 32, 128, 1, 128, [4000], 0, 4, 64, BF, False),
    "512 channels, one CTA a query": (100, 1, 64, 512, 4, 128, [600] * 100, 130, 4, 64, BF, True),
    "512 channels, a cluster": (1, 1, 64, 512, 4, 128, [3000], 500, 8, 64, BF, True),
    "one CTA a query, no sink": (100, 1, 16, 128, 4, 64, [500] * 100, 40, 4, 16, BF, False),
    "512 channels, one CTA a query, no sink": (100, 1, 64, 512, 4, 128, [600] * 100, 130, 4, 64, BF, False),
    "512 channels, few heads": (2, 1, 8, 512, 4, 128, [3000, 5], 500, 4, 64, BF, True),
}


@pytest.mark.parametrize("name", CASES)
def test_attention_gives_up_and_the_next_call_is_correct(name):
    case = CASES[name]
    b, s_q, H, d = case[:4]
    parts = attn_case(np.random.default_rng(7), case)
    o, lse = run_attn(case, parts)
    assert csa.csa_get_device_status(with_site=True) == (0, 0)
    n = b * s_q * H
    big_o = torch.full((n + 2, d), 7.0, dtype=BF, device="cuda")
    big_l = torch.full((n + 8,), 7.0, device="cuda")
    got = with_armed(SITE_ATTN, lambda: run_attn(case, parts, out=big_o[1:-1].view(b, s_q, H, d),
                                                 lse=big_l[4:-4].view(b, s_q, H)))
    assert got == (CSA_ERR_TIMEOUT, SITE_ATTN), got
    assert bool((big_o[0] == 7).all()) and bool((big_o[-1] == 7).all())
    assert bool((big_l[:4] == 7).all()) and bool((big_l[-4:] == 7).all())
    o2, lse2 = run_attn(case, parts)
    assert csa.csa_get_device_status(with_site=True) == (0, 0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fill", [0, 0xFF, 0x7F])
@pytest.mark.parametrize("b,s_q,n,topk", [(1, 1, 1000, 50), (2, 2, 3000, 300), (1, 1, 40000, 512), (1, 1, 300000, 700)])
def test_indexer_gives_up_and_the_next_call_is_correct(b, s_q, n, topk, fill):
    """The select then reads scores that were never written: whatever the workspace holds, it ends,
    and the indices that it writes are visible blocks."""
    page = 64
    cache, table, keys, q, w = index_case(np.random.default_rng(n), b, s_q, 16, 64, 1, [n] * b, 4, page, BF)
    q, w, table, lens = q.cuda(), w.cuda(), dev(table), dev([n] * b, torch.int32)
    want = serve.csa_indexer_topk_decode(q, cache, table, w, lens, topk, 1, page, 4)
    ws = torch.full((serve.csa_indexer_topk_decode_workspace_size(b, s_q, 16, 64, table.shape[1] * page),), fill,
                    dtype=torch.uint8, device="cuda")
    big = torch.full((b * s_q * topk + 16,), -7, dtype=torch.int32, device="cuda")
    out = big[8:-8].view(b, s_q, topk)
    got = with_armed(SITE_INDEX, lambda: serve.csa_indexer_topk_decode(q, cache, table, w, lens, topk, 1, page, 4,
                                                                       workspace=ws, out_idx=out))
    assert got == (CSA_ERR_TIMEOUT, SITE_INDEX), got
    assert bool((big[:8] == -7).all()) and bool((big[-8:] == -7).all())
    assert bool((((out >= 0) & (out < n)) | (out == -7)).all())
    again = serve.csa_indexer_topk_decode(q, cache, table, w, lens, topk, 1, page, 4, workspace=ws)
    assert csa.csa_get_device_status(with_site=True) == (0, 0)
    assert torch.equal(again, want)
