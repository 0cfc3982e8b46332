"""The serving calls' Python binding on the GPU: what it allocates, and calls whose
first one in a process is captured."""
import subprocess
import sys

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


FIRST_CALLS = """
import sys
sys.path[:0] = {path!r}
import torch
from compressed_sparse_attention_sum_gb300 import csa, serve
g = torch.Generator(device="cuda").manual_seed(0)
b, n, page, bits, d = 3, 2000, 64, 4, {d}
P = -(-n // page)
cache = torch.zeros(b * P, serve.csa_cache_page_bytes(page, d, bits), dtype=torch.uint8, device="cuda")
icache = torch.zeros(b * P, serve.csa_cache_page_bytes(page, 128, bits), dtype=torch.uint8, device="cuda")
table = torch.arange(b * P, dtype=torch.int32, device="cuda").view(b, P)
rows = torch.randn(b, n, d, generator=g, device="cuda").bfloat16()
keys = torch.randn(b, n, 128, generator=g, device="cuda").bfloat16()
q = torch.randn(b, 1, {H}, d, generator=g, device="cuda").bfloat16()
q_I = torch.randn(b, 1, 64, 128, generator=g, device="cuda").bfloat16()
w = torch.randn(b, 1, 64, generator=g, device="cuda")
sink = torch.randn({H}, generator=g, device="cuda")
zero = torch.zeros(b, dtype=torch.int32, device="cuda")
lens = zero + n
def step():
    serve.csa_cache_write(rows, cache, table, zero, page, bits)
    serve.csa_cache_write(keys, icache, table, zero, page, bits)
    idx = serve.csa_indexer_topk_decode(q_I, icache, table, w, lens, 200, 1, page, bits)
    some = serve.csa_attn_decode(q, cache, table, table, idx, sink, lens, d ** -0.5, 1, 128, page, bits)
    every = serve.csa_attn_decode(q, cache, table, table, None, sink, lens, d ** -0.5, 1, 128, page, bits)
    return idx, *some, *every
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


@pytest.mark.parametrize("d,H", [(128, 32), (512, 64)])
def test_the_first_calls_of_a_process_can_be_captured(d, H):
    from compressed_sparse_attention_sum_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(path=sys.path, d=d, H=H)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
