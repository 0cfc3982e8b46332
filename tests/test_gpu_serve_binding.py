"""The serving calls' Python binding on the GPU: what it allocates."""
import numpy as np
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from compressed_sparse_attention_sum_gb300 import serve
from test_gpu_serve import BF, attn_case, dev, index_case, run_attn

pytestmark = pytest.mark.gpu


class Allocations(TorchDispatchMode):
    """Records the shapes of the tensors that operators return."""

    def __init__(self):
        super().__init__()
        self.shapes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if isinstance(out, torch.Tensor):
            self.shapes.append(tuple(out.shape))
        return out


def test_a_dispatch_mode_sees_every_output_and_workspace():
    from compressed_sparse_attention_sum_gb300 import build
    build.build()
    case = (2, 1, 32, 128, 4, 64, [500, 300], 50, 4, 16, BF, True)
    parts = attn_case(np.random.default_rng(1), case)
    cache, table, keys, q, w = index_case(np.random.default_rng(2), 2, 1, 64, 128, 4, [500, 300], 4, 16, BF)
    args = (q.cuda(), cache, dev(table), w.cuda(), dev([500, 300], torch.int32), 50, 4, 16, 4)
    want_i, want_a = serve.csa_indexer_topk_decode(*args), run_attn(case, parts)
    with Allocations() as seen:
        idx, (o, lse) = serve.csa_indexer_topk_decode(*args), run_attn(case, parts)
    for t in (idx, o, lse):
        assert tuple(t.shape) in seen.shapes
    assert (serve.csa_attn_decode_workspace_size(2, 1, 32, 128, 64, 50),) in seen.shapes
    assert torch.equal(idx, want_i) and torch.equal(o, want_a[0]) and torch.equal(lse, want_a[1])
