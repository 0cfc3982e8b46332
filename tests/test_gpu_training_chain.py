"""A training step of a layer whose rows are normalised and turned: csa_norm_rope of the queries and the raw rows,
csa_compress_norm_rope, csa_attn_fwd, csa_rope back, and the gradients of all of them in a row, against fp64
autograd through the same chain at the values that the calls made."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_sum_gb300 import csa, rows
from oracle import rows_oracle as orc
from test_gpu_row_calls import BF, EPS, F32, I32, close, f64

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


def selection(g, b, sq, n_c, K, ratio):
    """Up to K visible blocks of every query, ascending, then -1."""
    idx = torch.full((b, sq, K), -1, dtype=I32)
    for i in range(b):
        for t in range(sq):
            n = min((t + 1) // ratio, n_c)
            pick = torch.randperm(n, generator=g)[:K].sort().values
            idx[i, t, :len(pick)] = pick.int()
    return idx


def turned(x, f, half, back=False):
    """fp64 rows [b, s, H, d] whose last channels turn by the token's index."""
    u, v = (torch.tensor(i) for i in orc.pairs(2 * len(f), x.shape[-1] - 2 * len(f), half))
    a = (torch.arange(x.shape[1], dtype=torch.float64)[:, None] * torch.tensor(f))[:, None]
    c, s = a.cos(), a.sin() * (-1 if back else 1)
    y = x.clone()
    y[..., u], y[..., v] = x[..., u] * c - x[..., v] * s, x[..., u] * s + x[..., v] * c
    return y


def normed(x, kind, w):
    m = x.mean(-1, keepdim=True) if kind == orc.LAYER else 0
    return (x - m) / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + EPS) * w


class At(torch.autograd.Function):
    """The value that a call made, with the gradient of what it stands for."""

    @staticmethod
    def forward(ctx, formula, made):
        return made.double().cpu()

    @staticmethod
    def backward(ctx, g):
        return g, None


def bounds(q, kv, logits, probs, o, do, scale, dtype):
    """How far o, dq, dkv and dsink may be off (q, kv and do are what the calls had).

    r: half a step of the type, to which the tensor cores' probabilities, their gradients and o are rounded once (bf16); U = 2^-24.
    A logit, a dot product of fp32 sums: D U of its terms' magnitudes; a probability by that, by the same of the log-sum, and by
    some roundings of the exponential (rho, relative).  do.o takes o as it was rounded."""
    r, U = (2.0 ** -8 if dtype is BF else 0.0), orc.U
    dot = orc.D * U
    size = torch.einsum("bthd,bnd->bthn", q.abs(), kv.abs()) * scale
    e_s = dot * size.masked_fill(logits.isinf(), 0.0)
    p, sink = probs[..., :-1], probs[..., -1:]
    top = e_s.amax(-1, keepdim=True) + 80 * U
    rho = e_s + top
    e_o = torch.einsum("bthn,bnd->bthd", p * (rho + r + dot), kv.abs()) + max(r, U) * o.abs()
    e_D = (do.abs() * (e_o + dot * o.abs())).sum(-1, keepdim=True)
    dp = torch.einsum("bthd,bnd->bthn", do, kv)
    e_dp = dot * torch.einsum("bthd,bnd->bthn", do.abs(), kv.abs())
    D = (do * o).sum(-1, keepdim=True)
    ds = p * (dp - D)
    e_ds = (p * (rho * (dp - D).abs() + e_dp + e_D) + (r + 4 * U) * ds.abs()) * (1 + r)
    e_dq = scale * torch.einsum("bthn,bnd->bthd", e_ds + dot * ds.abs(), kv.abs())
    chain = q.shape[1] * q.shape[2] * U                 # additions of a row's shares, one after another
    e_dkv = torch.einsum("bthn,bthd->bnd", p * (rho + r + chain), do.abs()) + scale * torch.einsum("bthn,bthd->bnd", e_ds + chain * ds.abs(), q.abs())
    e_sink = (sink * ((top + chain) * D.abs() + e_D)).sum((0, 1))[:, 0]
    return e_o, e_dq, e_dkv, e_sink


@pytest.mark.parametrize("dtype,b,sq,H,d,half,kind", [(BF, 2, 70, 32, 128, False, orc.RMS), (BF, 1, 48, 64, 512, False, orc.RMS),
                                                       (F32, 2, 45, 4, 64, True, orc.LAYER), (BF, 1, 33, 8, 64, True, orc.RMS)])
def test_a_training_step(dtype, b, sq, H, d, half, kind):
    g = torch.Generator().manual_seed(d + sq)
    ratio, K, window, dim = 4, 5, 13, d // 2
    n_c, scale = sq // ratio, d ** -0.5
    draw = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    xq, xk, ckv, cscore, dz = draw(b, sq, H, d), draw(b, sq, d), draw(b, sq, d), draw(b, sq, d), draw(b, sq, H, d)
    wq, wk, wc = ((0.5 + torch.rand(d, generator=g)).cuda() for _ in range(3))
    sink, idx = torch.randn(H, generator=g).cuda(), selection(g, b, sq, n_c, K, ratio)
    layout = "half" if half else "interleaved"
    f = orc.freqs(dim)
    rope = rows.CsaRope(rows.csa_rope_turns(f), d - dim, layout)
    on_gpu = idx.cuda()

    def step():
        q = rows.csa_norm_rope(xq, kind, rope, None, wq, None, EPS)
        kv = torch.empty(b, sq + n_c, d, dtype=dtype, device="cuda")
        rows.csa_norm_rope(xk, kind, rope, None, wk, None, EPS, out=kv[:, :sq])
        csa.csa_compress_norm_rope(ckv, cscore, ratio, wc, EPS, dim, 40000.0, out=kv[:, sq:])
        o, lse = csa.csa_attn_fwd(q, kv, on_gpu, sink, scale, ratio, window)
        z = rows.csa_rope(o, rope, inverse=True)
        do = rows.csa_rope_bwd(dz, rope, inverse=True)
        dq, dkv, dsink = csa.csa_attn_bwd(q, kv, on_gpu, sink, scale, ratio, window, o, lse, do)
        dxq, dwq, _ = rows.csa_norm_rope_bwd(xq, dq, kind, rope, None, wq, EPS)
        dxk, dwk, _ = rows.csa_norm_rope_bwd(xk, dkv[:, :sq], kind, rope, None, wk, EPS)
        return q, kv, o, z, do, dq, dkv, dsink, dxq, dwq, dxk, dwk

    def check(q, kv, o, z, do, dq, dkv, dsink, dxq, dwq, dxk, dwk):
        leaves = [torch.tensor(f64(t), requires_grad=True) for t in (xq, wq, xk, wk, sink)]
        q64 = At.apply(turned(normed(leaves[0], kind, leaves[1]), f, half), q)
        raw = At.apply(turned(normed(leaves[2], kind, leaves[3])[:, :, None], f, half)[:, :, 0], kv[:, :sq])
        blocks = torch.tensor(f64(kv[:, sq:]), requires_grad=True)
        kv64 = torch.cat((raw, blocks), 1)
        t, s = torch.arange(sq)[:, None], torch.arange(sq)[None]
        seen = torch.zeros(b, sq, sq + n_c, dtype=torch.bool)
        seen[:, :, :sq] = (s <= t) & (s > t - window)
        for k in range(K):
            i, at = (idx[..., k] >= 0).nonzero(as_tuple=True)
            seen[i, at, sq + idx[i, at, k].long()] = True
        logits = torch.einsum("bthd,bnd->bthn", q64, kv64) * scale
        logits = logits.masked_fill(~seen[:, :, None], float("-inf"))
        probs = torch.softmax(torch.cat((logits, leaves[4].expand(b, sq, H)[..., None]), -1), -1)
        p = probs[..., :-1]
        o64 = torch.einsum("bthn,bnd->bthd", p, kv64)
        z64 = turned(At.apply(o64, o), f, half, back=True)
        pos = np.broadcast_to(np.arange(sq)[:, None], (b, sq, H))
        close(z, f64(z64), orc.turn(f64(o), pos, f, d - dim, half, 1.0, back=True)[1])
        # the gradient of o is rounded to its type once: autograd goes on from that
        seed, = torch.autograd.grad(z64, o64, dz.double().cpu(), retain_graph=True)
        close(do, f64(seed), orc.turn(f64(dz), pos, f, d - dim, half, 1.0)[1])
        got = torch.autograd.grad(o64, [q64, raw, blocks, *leaves], do.double().cpu())
        e_o, e_dq, e_dkv, e_ds = bounds(*(v.detach() for v in (q64, kv64, logits, probs, o64)), do.double().cpu(), scale, dtype)
        for mine, want, e, what in ((o, o64.detach(), e_o, "o"), (dq, got[0], e_dq, "dq"), (dkv[:, :sq], got[1], e_dkv[:, :sq], "dkv"),
                                    (dkv[:, sq:], got[2], e_dkv[:, sq:], "blocks"), (dsink, got[7], e_ds, "dsink")):
            off = ((mine.double().cpu() - want).abs() / (e + 1e-30)).max().item()
            assert off <= 1, (what, off)
        # the turn and the norm spread these errors as they spread any
        for x, w, dy, e, dx, dw, ref in ((xq, wq, got[0], e_dq, dxq, dwq, got[3:5]),
                                         (xk[:, :, None], wk, got[1][:, :, None], e_dkv[:, :sq, None], dxk[:, :, None], dwk, got[5:7])):
            at = np.broadcast_to(np.arange(sq)[:, None], x.shape[:3])
            back, eb = orc.turn(f64(dy), at, f, d - dim, half, 1.0, back=True)
            eb = eb + orc.spread(f64(e), f, d - dim, half, 1.0)
            want, err = orc.norm_bwd(f64(x).reshape(-1, d), back.reshape(-1, d), eb.reshape(-1, d), kind, f64(w), EPS)
            r0, r1 = f64(ref[0]).reshape(-1, d), f64(ref[1])
            assert np.abs(want[0] - r0).max() <= 1e-9 * np.abs(r0).max() and np.abs(want[1] - r1).max() <= 1e-9 * np.abs(r1).max()
            close(dx.reshape(-1, d), want[0], err[0])
            close(dw, want[1], err[1])
            # ... and they are those of what the attention gave
            dy = dq if x is xq else dkv[:, :sq, None]
            back, eb = orc.turn(f64(dy), at, f, d - dim, half, 1.0, back=True)
            want, err = orc.norm_bwd(f64(x).reshape(-1, d), back.reshape(-1, d), eb.reshape(-1, d), kind, f64(w), EPS)
            close(dx.reshape(-1, d), want[0], err[0])
            close(dw, want[1], err[1])

    check(*step())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        made = step()
    for t in (xq, xk, dz):                              # other inputs in the same places
        t.copy_(draw(*t.shape))
    graph.replay()
    torch.cuda.synchronize()
    check(*made)
