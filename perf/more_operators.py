"""Workloads of the calls that make a CSA layer's rows: layer and RMS norms, rotary
positions, both in one pass, and the compressor for the newest tokens of a sequence.

Each case is one call as a training step, a prompt or a decode step makes it, in a
plain form of elementary torch operations (`own` false) and through the library's
entry points (`own` true).  All inputs are synthetic; the head layouts are those of
the repository's workloads (CSA-4, HCA, production width), the widths of whole
token rows are generic.

Rotation: pair i of the `rope` channels from `first` on turns by pos * freq[i];
interleaved pairs are neighbours, half pairs lie rope / 2 apart.  Long contexts
scale the frequencies by parts (low ones divided by the factor, high ones kept) and
the turned channels by 0.1 ln(factor) + 1.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
GOLD = 0.6180339887498949


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch's token rows before a layer (latency)
        dict(name="norm_token", op="norm", rows=16, n=4096, kind="rms", affine=True, fp32=False, pad=0),
        # the token rows of two long prompts, layer norm with weight and bias
        dict(name="norm_layer_prompt", op="norm", rows=16384, n=4096, kind="layer", affine=True, fp32=False, pad=0),
        # a training step's gradient of wide token rows, with the weight's and the bias's sums
        dict(name="norm_layer_bwd", op="norm_bwd", rows=8191, n=7168, kind="layer", affine=True, fp32=False, grad32=False, pad=0),
        # fp32 rows of an odd width that lie inside wider ones (a slice of a fused projection)
        dict(name="norm_rms_bwd_fp32", op="norm_bwd", rows=1021, n=2056, kind="rms", affine=True, fp32=True, grad32=True, pad=24),
        # queries of a decode batch at the production width, far positions, 64 of 512 channels, scaled for a long context
        dict(name="rope_token_d512", op="rope", b=64, s=1, H=64, d=512, rope=64, first=448, half=False, long=True, extra=0, fp32=False,
             inverse=False, far=1000000),
        # a ragged pair of prompts, half layout over the whole head, queries inside a fused projection
        dict(name="rope_prompt_half", op="rope", b=2, s=4097, H=32, d=128, rope=128, first=0, half=True, long=False, extra=2, fp32=False,
             inverse=False, far=0),
        # the attention's fp32 query gradient turned back, production width
        dict(name="rope_bwd_d512", op="rope_bwd", b=1, s=4096, H=64, d=512, rope=64, first=448, half=False, long=False, extra=0, fp32=True,
             out32=False, inverse=False, far=0),
        # CSA-4 queries of a decode batch with a draft token each (latency)
        dict(name="norm_rope_token", op="norm_rope", b=16, s=2, H=32, d=128, rope=64, first=64, half=False, long=False, extra=0, kind="rms",
             fp32=False, far=131072),
        # production width: the queries of two prompts (HBM)
        dict(name="norm_rope_prompt_d512", op="norm_rope", b=2, s=8192, H=64, d=512, rope=64, first=448, half=False, long=True, extra=0,
             kind="rms", fp32=False, far=0),
        # CSA-4 training step: the attention's fp32 gradient through rotation and norm, weight's sum over all heads
        dict(name="norm_rope_bwd", op="norm_rope_bwd", b=1, s=4096, H=32, d=128, rope=128, first=0, half=True, long=False, extra=0,
             kind="rms", fp32=False, grad32=True, far=0),
        # a decode batch of the production width with overlapping blocks; a quarter of the sequences complete one
        dict(name="compress_token_d512", op="compress", b=96, s=1, d=512, ratio=4, coff=2, wide=True, rope=64, kind="rms", long=True,
             max_len=65536, pad=2),
        # the next 2000 tokens of three HCA prompts, blocks of 128 that began in the rows before
        dict(name="compress_chunk_hca", op="compress", b=3, s=2000, d=128, ratio=128, coff=1, wide=True, rope=64, kind="rms", long=False,
             max_len=100000, pad=0),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_rope(rng, d):
    """Turned channels of a head of d: a whole head, a half, a small part; at its start or its end."""
    half = rng.random() < 0.5
    rope = rng.choice([d, d // 2, 32, 64, 24 if half else 22])
    rope = min(d, rope - rope % (4 if half else 2))
    return dict(rope=rope, first=rng.choice([0, d - rope]), half=half, long=rng.random() < 0.3)


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "rope", "rope_bwd", "norm_rope", "norm_rope_bwd", "compress", "compress"])
    fp32 = rng.random() < 0.3
    if op.startswith("norm") and "rope" not in op:
        n = 8 * _spread(rng, 8, 2048)
        case = dict(op=op, rows=_spread(rng, 1, (1 << 25) // n), n=n, kind=rng.choice(["rms", "layer"]), affine=rng.random() < 0.8,
                    fp32=fp32, pad=rng.choice([0, 8, 136]))
        return dict(case, grad32=rng.random() < 0.5) if op == "norm_bwd" else case
    if op == "compress":
        d, ratio = rng.choice([64, 128, 128, 256, 512]), rng.choice([4, 4, 8, 128])
        b, s = _spread(rng, 1, 96), rng.choice([1, 1, 2, 5, 300])
        return dict(op=op, b=b if s < 300 else min(b, 8), s=s, d=d, ratio=ratio, coff=rng.choice([1, 2]), wide=rng.random() < 0.7,
                    rope=rng.choice([32, 64]), kind=rng.choice(["rms", "layer"]), long=rng.random() < 0.3,
                    max_len=_spread(rng, 40, 262144), pad=rng.choice([0, 1]))
    d, H, b = rng.choice([64, 80, 128, 128, 192, 512]), rng.choice([1, 3, 8, 32, 64]), rng.randint(1, 5)
    case = dict(op=op, b=b, s=_spread(rng, 1, max(1, (1 << 25) // (b * H * d))), H=H, d=d, **_draw_rope(rng, d), extra=rng.choice([0, 0, 2]),
                fp32=fp32, far=rng.choice([0, 0, 5000, 1000000]))
    if "norm" in op:
        case["kind"] = rng.choice(["rms", "layer"])
    if op == "norm_rope_bwd":
        case["grad32"] = rng.random() < 0.5
    if op.startswith("rope"):
        case["inverse"] = rng.random() < 0.3
    if op == "rope_bwd":
        case["out32"] = rng.random() < 0.5
    return case


def _lens(case):
    """Tokens of each sequence, the new ones included; the last `pad` have none."""
    n, top, s = case["b"], max(case["max_len"], case["s"]), case["s"]
    out = [top] + [s + int((top - s) * ((i * GOLD) % 1.0)) for i in range(1, n)]
    for i in range(max(1, n - case["pad"]), n):
        out[i] = 0
    return out


def _blocks(case):
    """(first block, blocks) that each sequence's new tokens complete."""
    return [(max(0, n - case["s"]) // case["ratio"], n // case["ratio"] - max(0, n - case["s"]) // case["ratio"]) for n in _lens(case)]


def work(case):
    op, e = case["op"], 4 if case.get("fp32") else 2
    if op in ("norm", "norm_bwd"):
        items, p = case["rows"] * case["n"], 4 * case["n"] * (2 if case["kind"] == "layer" else 1) * case["affine"]
        if op == "norm":
            return {"bytes": 2 * items * e + p, "flops": 6 * items}
        g = 4 if case["grad32"] else 2
        return {"bytes": items * (2 * e + g) + p + 4 * case["n"] * case["affine"], "flops": 14 * items}
    if op == "compress":
        done, new = sum(n for _, n in _blocks(case)), sum(min(case["s"], n) for n in _lens(case))
        old = 0                            # rows of the ring that the completed blocks read
        for n, (j, k) in zip(_lens(case), _blocks(case)):
            old += max(0, max(0, n - case["s"]) - max(0, (j + 1 - case["coff"]) * case["ratio"])) if k else 0
        w = case["d"] + (case["d"] if case["wide"] else 1)
        return {"bytes": 2 * (2 * new + old) * w + 2 * done * case["d"] + 8 * case["b"],
                "flops": done * case["d"] * (5 * case["coff"] * case["ratio"] + 10)}
    items = case["b"] * case["s"] * case["H"] * case["d"]
    if op in ("rope", "rope_bwd"):
        o = e if op == "rope" else 4 if case["out32"] else 2
        return {"bytes": items * (e + o) + 4 * case["b"] * case["s"] * (case["far"] > 0), "flops": 3 * items * case["rope"] // case["d"]}
    byts, p = items * 2 * e, 4 * case["d"] * (2 if case["kind"] == "layer" else 1)
    if op == "norm_rope_bwd":
        byts += items * (4 if case["grad32"] else 2) + 4 * case["d"]
    return {"bytes": byts + p + 4 * case["b"] * case["s"] * (case["far"] > 0), "flops": items * (14 if op == "norm_rope_bwd" else 6)}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 1000003 + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _rows(g, dtype, shape, width, pad=0):
    """Rows as projections give them: channels of different size and mean; every row `pad` channels apart."""
    scale = torch.exp(0.5 * _randn(g, width))
    shift = 0.3 * _randn(g, width)
    x = torch.empty(*shape[:-1], shape[-1] + pad, dtype=dtype, device=DEV)
    x.normal_(generator=g)
    y = x[..., :shape[-1]]
    y.unflatten(-1, (-1, width)).mul_(scale).add_(shift)
    return y


def _freqs(dim, base, long):
    """fp64 frequencies; `long`: a context of 4096 stretched 16 times, by parts."""
    i = torch.arange(dim // 2, dtype=torch.float64, device=DEV)
    f = base ** (-2 * i / dim)
    if long:
        lo, hi = (dim * math.log(4096 / (2 * math.pi * n)) / (2 * math.log(base)) for n in (32, 1))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), dim - 1)
        g = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - g) + f / 16 * g
    return f


def _turned(st, case, dim, first, half):
    """The rotation of a case: what the plain form takes, and the plan that a user's program keeps."""
    base = 40000.0 if case["op"] == "compress" else 10000.0
    st.update(freq=_freqs(dim, base, case["long"]), first=first, half=half,
              factor=0.1 * math.log(16) + 1 if case["long"] else 1.0)
    if own:
        from compressed_sparse_attention_sum_gb300 import rows
        f = rows.csa_rope_freqs(dim, base, "by_parts" if case["long"] else "plain", factor=16.0, original_len=4096.0)
        st["plan"] = rows.CsaRope(rows.csa_rope_turns(f, DEV), first, "half" if half else "interleaved", st["factor"])


def prepare(case, seed):
    g, op, st = _gen(seed), case["op"], dict(case)
    if op == "compress":
        return _prepare_compress(st, case, g)
    dtype = torch.float32 if case["fp32"] else torch.bfloat16
    if op in ("norm", "norm_bwd"):
        d = case["n"]
        st["x"] = _rows(g, dtype, (case["rows"], d), d, case["pad"])
    else:
        b, s, H, d = case["b"], case["s"], case["H"], case["d"]
        st["x"] = _rows(g, dtype, (b, s, H * d), d, case["extra"] * d).unflatten(-1, (H, d))
        st["pos"] = None
        if case["far"]:                    # every sequence continues at a place of its own
            at = [case["far"] - int(case["far"] * ((i * GOLD) % 1.0)) + seed % 7 for i in range(b)]
            st["pos"] = (torch.tensor(at, device=DEV)[:, None] + torch.arange(s, device=DEV)).int()
        _turned(st, case, case["rope"], case["first"], case["half"])
    st["weight"] = st["bias"] = None
    if case.get("affine", "kind" in case):
        st["weight"] = 1 + 0.2 * _randn(g, d)
        st["bias"] = 0.1 * _randn(g, d) if case["kind"] == "layer" else None
    if "bwd" in op and "norm" in op:
        st["dout"] = torch.empty(st["x"].shape, dtype=torch.float32 if case["grad32"] else torch.bfloat16, device=DEV).normal_(generator=g)
        if own:
            from compressed_sparse_attention_sum_gb300 import rows
            size = rows.csa_norm_bwd_workspace_size(st["x"].numel() // d, d, st["weight"] is not None, st["bias"] is not None)
            st["ws"] = torch.empty(max(16, size), dtype=torch.uint8, device=DEV)
    out = dtype
    if op == "rope_bwd":
        out = torch.float32 if case["out32"] else torch.bfloat16
    st["out"] = torch.empty(st["x"].shape, dtype=out, device=DEV)
    return st


def _prepare_compress(st, case, g):
    b, s, d, r, dtype = case["b"], case["s"], case["d"], case["ratio"], torch.bfloat16
    w, R = d if case["wide"] else 1, case["coff"] * r + s - 1
    st["kv"], st["score"] = _rows(g, dtype, (b, s, d), d), (_randn(g, b, s, w) * 1.5).to(dtype)
    st["kv_ring"], st["score_ring"] = _rows(g, dtype, (b, R, d), d), (_randn(g, b, R, w) * 1.5).to(dtype)
    st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
    st["weight"] = 1 + 0.2 * _randn(g, d)
    st["bias"] = 0.1 * _randn(g, d) if case["kind"] == "layer" else None
    st["out"] = torch.zeros(b, -(-s // r), d, dtype=dtype, device=DEV)
    t = st["lens"].long()[:, None] - s + torch.arange(s, device=DEV)
    st["at"], st["i"] = (t >= 0).nonzero(as_tuple=True)      # the new rows that are a token, and their places in the ring
    st["slot"] = t[st["at"], st["i"]] % R
    _turned(st, case, case["rope"], d - case["rope"], False)
    return st


# ------------------------------------------------------------------- run

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from compressed_sparse_attention_sum_gb300 import rows
    op = st["op"]
    kind = {"rms": rows.CSA_NORM_RMS, "layer": rows.CSA_NORM_LAYER}[st["kind"]] if "kind" in st else 0
    if op == "norm":
        return rows.csa_norm(st["x"], kind, st["weight"], st["bias"], EPS, out=st["out"])
    if op == "norm_bwd":
        return rows.csa_norm_bwd(st["x"], st["dout"], kind, st["weight"], EPS, has_bias=st["bias"] is not None, dx=st["out"],
                                 workspace=st["ws"])
    if op == "rope":
        return rows.csa_rope(st["x"], st["plan"], st["pos"], inverse=st["inverse"], out=st["out"])
    if op == "rope_bwd":
        return rows.csa_rope_bwd(st["x"], st["plan"], st["pos"], inverse=st["inverse"], dx=st["out"])
    if op == "norm_rope":
        return rows.csa_norm_rope(st["x"], kind, st["plan"], st["pos"], st["weight"], st["bias"], EPS, out=st["out"])
    if op == "norm_rope_bwd":
        return rows.csa_norm_rope_bwd(st["x"], st["dout"], kind, st["plan"], st["pos"], st["weight"], EPS,
                                      has_bias=st["bias"] is not None, dx=st["out"], workspace=st["ws"])
    out, first, counts = rows.csa_compress_decode(
        st["kv"], st["score"], st["kv_ring"], st["score_ring"], st["lens"], st["ratio"], st["coff"], kind, st["weight"], st["bias"], EPS,
        st["plan"], out=st["out"])
    return out, first, counts, st["kv_ring"], st["score_ring"]


def _normed(x, kind, weight, bias):
    """(norm, normalised rows, 1 / deviation) of fp32 rows."""
    c = x - x.mean(-1, keepdim=True) if kind == "layer" else x
    r = torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
    xh = c * r
    y = xh if weight is None else xh * weight
    return y if bias is None else y + bias, xh, r


def _normed_grad(x, g, kind, weight):
    """(dx, dweight, dbias) of fp32 rows and fp32 gradients."""
    _, xh, r = _normed(x, kind, None, None)
    gw = g if weight is None else g * weight
    dx = gw - xh * (gw * xh).mean(-1, keepdim=True)
    if kind == "layer":
        dx = dx - gw.mean(-1, keepdim=True)
    return dx * r, (g * xh).flatten(0, -2).sum(0), g.flatten(0, -2).sum(0)


def _turn(st, x, pos, back=False):
    """fp32 rows [b, s, H, d] turned by their token's position [b or 1, s] (angles in 64 bits)."""
    n, at = 2 * len(st["freq"]), st["first"]
    a = pos.double()[..., None, None] * st["freq"]
    c, s = a.cos().float() * st["factor"], a.sin().float() * (-st["factor"] if back else st["factor"])
    y, z = x.clone(), x[..., at:at + n]
    u, v = (z[..., :n // 2], z[..., n // 2:]) if st["half"] else (z[..., 0::2], z[..., 1::2])
    p, q = u * c - v * s, u * s + v * c
    y[..., at:at + n] = torch.cat((p, q), -1) if st["half"] else torch.stack((p, q), -1).flatten(-2)
    return y


def _run_plain(st):
    op = st["op"]
    if op == "compress":
        return _compress_plain(st)
    x = st["x"].float()
    if op == "norm":
        return _normed(x, st["kind"], st["weight"], st["bias"])[0].to(st["x"].dtype)
    if op == "norm_bwd":
        g, dtype = st["dout"].float(), st["out"].dtype
        dx, dw, db = _normed_grad(x, g, st["kind"], st["weight"])
        return dx.to(dtype), None if st["weight"] is None else dw, None if st["bias"] is None else db
    pos = st["pos"] if st["pos"] is not None else torch.arange(x.shape[1], device=DEV)[None]
    if op in ("rope", "rope_bwd"):
        return _turn(st, x, pos, back=st["inverse"] != (op == "rope_bwd")).to(st["out"].dtype)
    if op == "norm_rope":
        return _turn(st, _normed(x, st["kind"], st["weight"], st["bias"])[0], pos).to(st["x"].dtype)
    dx, dw, db = _normed_grad(x, _turn(st, st["dout"].float(), pos, back=True), st["kind"], st["weight"])
    return dx.to(st["out"].dtype), dw, None if st["bias"] is None else db


def _compress_plain(st):
    r, coff, s, R = st["ratio"], st["coff"], st["s"], st["kv_ring"].shape[1]
    lens = st["lens"].long()
    t0 = (lens - s)[:, None, None]
    first = (lens - s).clamp_min(0) // r
    counts = lens // r - first
    j = first[:, None] + torch.arange(st["out"].shape[1], device=DEV)                         # [b, blocks]
    p = (j[..., None] + 1 - coff) * r + torch.arange(coff * r, device=DEV)                     # positions that each pools
    from_ring = torch.remainder(p, R)
    src = torch.where(p >= t0, R + (p - t0).clamp_max(s - 1), from_ring)
    bi = torch.arange(len(lens), device=DEV)[:, None, None]
    kv = torch.cat((st["kv_ring"], st["kv"]), 1)[bi, src].float()                              # [b, blocks, tokens, d]
    z = torch.cat((st["score_ring"], st["score"]), 1)[bi, src].float()
    z = torch.where(p[..., None] >= 0, z, torch.full_like(z, -math.inf))
    e = torch.exp(z - z.amax(2, keepdim=True))
    pooled = ((e * kv).sum(2) / e.sum(2)).to(st["kv"].dtype).float()
    y = _normed(pooled, st["kind"], st["weight"], st["bias"])[0]
    y = _turn(st, y[:, :, None], (j + 1) * r - 1)[:, :, 0].to(st["out"].dtype)
    live = torch.arange(st["out"].shape[1], device=DEV) < counts[:, None]
    st["kv_ring"][st["at"], st["slot"]] = st["kv"][st["at"], st["i"]]
    st["score_ring"][st["at"], st["slot"]] = st["score"][st["at"], st["i"]]
    return torch.where(live[..., None], y, st["out"]), first.int(), counts.int(), st["kv_ring"], st["score_ring"]


# ----------------------------------------------------------------- exact

def _unit(x, kind, weight, bias):
    """The norm's definition."""
    if kind == "layer":
        y = (x - x.mean(-1, True)) / torch.sqrt(x.var(-1, correction=0, keepdim=True) + EPS)
    else:
        y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    if weight is not None:
        y = y * weight.double()
    return y if bias is None else y + bias.double()


def _spun(st, x, pos):
    """The rotation's definition: pairs as complex numbers, times scale * exp(i pos freq); x [..., H, d], pos [..., 1] or alike."""
    n, at = 2 * len(st["freq"]), st["first"]
    angle = pos.double()[..., None, None] * st["freq"]
    by = torch.polar(torch.full_like(angle, st["factor"]), angle)
    z = x[..., at:at + n]
    pair = (2, n // 2) if st["half"] else (n // 2, 2)
    z = z.unflatten(-1, pair)
    z = z.transpose(-1, -2) if st["half"] else z
    w = torch.view_as_real(torch.view_as_complex(z.contiguous()) * by)
    w = (w.transpose(-1, -2) if st["half"] else w).flatten(-2)
    return torch.cat((x[..., :at], w, x[..., at + n:]), -1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "compress":
        return _exact_compress(st)
    x = st["x"].double()
    if op == "norm":
        return _unit(x, case["kind"], st["weight"], st["bias"])
    if "norm" not in op or op == "norm_rope":
        pos = st["pos"] if st["pos"] is not None else torch.arange(x.shape[1], device=DEV)[None]
        if op == "norm_rope":
            return _spun(st, _unit(x, case["kind"], st["weight"], st["bias"]), pos)
        return _spun(st, x, -pos if case["inverse"] != (op == "rope_bwd") else pos)
    x = x.detach().requires_grad_()
    w = None if st["weight"] is None else st["weight"].double().requires_grad_()
    c = None if st["bias"] is None else st["bias"].double().requires_grad_()
    y = _unit(x, case["kind"], w, c)
    if op == "norm_rope_bwd":
        y = _spun(st, y, st["pos"] if st["pos"] is not None else torch.arange(x.shape[1], device=DEV)[None])
    wanted = [t for t in (x, w, c) if t is not None]
    got = dict(zip(map(id, wanted), torch.autograd.grad(y, wanted, st["dout"].double())))
    return got[id(x)], got.get(id(w)), got.get(id(c))


def _exact_compress(st):
    r, s, R, d = st["ratio"], st["s"], st["kv_ring"].shape[1], st["d"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    first, counts = (torch.zeros(st["b"], dtype=torch.int32, device=DEV) for _ in range(2))
    rings = [st["kv_ring"].clone(), st["score_ring"].clone()]
    for i, n in enumerate(st["lens"].tolist()):
        begin = max(0, n - s)
        for p in range(begin, n):
            for ring, new in zip(rings, (st["kv"], st["score"])):
                ring[i, p % R] = new[i, p - (n - s)]
        first[i], counts[i] = begin // r, n // r - begin // r
        for k, j in enumerate(range(begin // r, n // r)):
            ps = torch.arange(max(0, (j + 1 - st["coff"]) * r), (j + 1) * r, device=DEV) % R
            weights = torch.softmax(rings[1][i, ps].double(), 0)
            pooled = (weights * rings[0][i, ps].double()).sum(0).to(st["kv"].dtype).double()
            y = _unit(pooled, st["kind"], st["weight"], st["bias"])
            out[i, k] = _spun(st, y[None], torch.tensor((j + 1) * r - 1, device=DEV))[0]
    return out, first, counts, rings[0].double(), rings[1].double()
