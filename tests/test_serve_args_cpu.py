"""Arguments of the serving calls on the host (no GPU needed): what is refused before
any CUDA call, beyond test_serve_cpu.py."""
import itertools

import pytest

from compressed_sparse_attention_sum_gb300 import build, serve
from test_serve_cpu import INVALID, UNSUPPORTED, _read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return serve.load_library()


def test_rows_of_a_read_that_share_elements_are_refused(lib):
    """Every pair of strides of 2 to 4 sequences of 2 to 5 rows, against the rows' own ranges.
    P is beyond the limit, so that what is not refused for its strides is UNSUPPORTED."""
    d = 32
    seen = set()
    for b, s, bs, rs in itertools.product((2, 3, 4), (2, 3, 5), range(32, 208, 16), range(32, 208, 16)):
        taken = [set(range(i * bs + j * rs, i * bs + j * rs + d)) for i in range(b) for j in range(s)]
        shared = len(set().union(*taken)) < d * len(taken)
        got = _read(lib, b=b, s=s, d=d, bs=bs, rs=rs, P=1 << 19)
        assert got == (INVALID if shared else UNSUPPORTED), (b, s, bs, rs)
        seen.add(shared)
    assert seen == {True, False}


def test_no_attention_workspace_exceeds_the_stated_bound(lib):
    """... and it does shrink as a batch grows, so the largest batch's size is not the bound."""
    size = lib.csa_attn_decode_workspace_size
    for d, H in itertools.product((32, 64, 96, 512), (1, 7, 8, 16, 32, 33, 64, 96, 128)):
        for b, s_q in itertools.product((1, 2, 3, 5, 8, 11, 12, 13, 24, 36, 64, 76, 144, 152, 304, 400), (1, 2, 3, 4, 7)):
            for window, rows in itertools.product((1, 128), (0, 512, 1100, 1 << 20)):
                assert size(b, s_q, H, d, window, rows) <= 2880 * (4 * d + 8) + 16, (d, H, b, s_q, window, rows)
    assert size(8, 1, 32, 128, 128, 512) > size(64, 1, 32, 128, 128, 512) == 0
