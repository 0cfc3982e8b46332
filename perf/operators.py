"""Workloads of the serving operators of a CSA layer: the quantised paged cache
(write, read), the single-token indexer and the single-token attention.

Each case is one operator's call as a decode step (or a prompt) makes it, in a
plain form of elementary torch operations (`own` false) and through the
library's entry points (`own` true).  All sizes are synthetic; the layer widths
are those of the repository's workloads (CSA-4, HCA, production width).

Cache: pages of `page` rows; a page holds page x (d * bits / 8) bytes of codes,
then page x (d / 32) scale bytes.  A group of 32 channels is codes times
2^(byte - 127); bits 4: e2m1 codes, channel 2i in the low half of byte i; bits
8: e4m3 codes.  Position p of a sequence lies in slot p mod (P * page) of its
row of the page table [b, P].
"""
import math

import torch

own = False

GROUP = 32
MIN_EXP = -110            # smallest scale exponent
TOP = {4: 6.0, 8: 448.0}  # largest code value
RATIO_GOLD = 0.6180339887498949
DEV = "cuda"


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's rows of eight sequences into the CSA-4 layer's 4-bit cache (latency)
        dict(name="write_token", op="write", b=8, s=1, d=128, bits=4, page=64, ragged=False, fp32=False),
        # two prompts of the production width into a 4-bit cache
        dict(name="write_prompt_d512", op="write", b=2, s=8192, d=512, bits=4, page=64, ragged=False, fp32=False),
        # ragged fp32 rows (an fp32 compressor's output) into an 8-bit cache, pages that end inside a sequence
        dict(name="write_ragged_8bit", op="write", b=5, s=4097, d=128, bits=8, page=48, ragged=True, fp32=True),
        # the window rows of four sequences read back before a prompt is continued
        dict(name="read_window_8bit", op="read", b=4, s=131, d=128, bits=8, page=64, ragged=True, fp32=False),
        # the compressed rows of two long sequences of the production width read back
        dict(name="read_long_d512", op="read", b=2, s=32768, d=512, bits=4, page=64, ragged=False, fp32=False),
        # one sequence at 4096 tokens: the CSA-4 indexer for its next token
        dict(name="index_b1", op="index", b=1, s_q=1, H_I=64, d_I=128, ratio=4, topk=512, max_len=4096, bits=4, page=64, pad=0),
        # a decode batch of ragged lengths up to 128 Ki tokens
        dict(name="index_b16_long", op="index", b=16, s_q=1, H_I=64, d_I=128, ratio=4, topk=512, max_len=131072, bits=4, page=64, pad=1),
        # two draft tokens a sequence, 8-bit index keys, 1024 selected
        dict(name="index_draft_8bit", op="index", b=6, s_q=2, H_I=64, d_I=128, ratio=4, topk=1024, max_len=50001, bits=8, page=48, pad=0),
        # CSA-4 layer, one sequence (latency)
        dict(name="attend_b1", op="attend", b=1, s_q=1, H=32, d=128, ratio=4, window=128, topk=512, max_len=4096, bits=4, page=64, pad=0),
        # CSA-4 layer, a ragged decode batch with two empty places, 8-bit cache
        dict(name="attend_b64_8bit", op="attend", b=64, s_q=1, H=32, d=128, ratio=4, window=128, topk=512, max_len=40000, bits=8, page=64, pad=2),
        # production width, 128 sequences, 4-bit cache
        dict(name="attend_b128_d512", op="attend", b=128, s_q=1, H=64, d=512, ratio=4, window=128, topk=1024, max_len=16384, bits=4, page=64, pad=0),
        # HCA layer: every visible block of a million tokens, two draft tokens
        dict(name="attend_hca", op="attend", b=4, s_q=2, H=32, d=128, ratio=128, window=128, topk=0, max_len=1048576, bits=4, page=64, pad=0),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "index", "attend", "index", "attend"])
    bits, page = rng.choice([4, 8]), rng.choice([16, 48, 64, 128])
    if op in ("write", "read"):
        d, b = rng.choice([64, 128, 256, 512]), rng.randint(1, 9)
        return dict(op=op, b=b, s=_spread(rng, 1, 8 * 1024 * 1024 // (d * b)), d=d, bits=bits, page=page,
                    ragged=rng.random() < 0.5, fp32=rng.random() < 0.3)
    if op == "index":
        b, s_q = _spread(rng, 1, 24), rng.choice([1, 1, 2, 3])
        return dict(op=op, b=b, s_q=s_q, H_I=rng.choice([8, 32, 64]), d_I=rng.choice([64, 128]), ratio=4,
                    topk=rng.choice([64, 256, 512, 1024]), max_len=_spread(rng, 300, 1048576 // (b * s_q)), bits=bits, page=page,
                    pad=rng.choice([0, 0, 1]) if b > 1 else 0)
    b, s_q, d = _spread(rng, 1, 96), rng.choice([1, 1, 2, 4]), rng.choice([64, 128, 128, 512])
    hca = rng.random() < 0.3
    return dict(op=op, b=b, s_q=s_q if b < 25 else 1, H=rng.choice([8, 16, 32, 64]), d=d, ratio=128 if hca else 4, window=rng.choice([31, 128]),
                topk=0 if hca else rng.choice([64, 512, 1024]), max_len=_spread(rng, 130, 262144 if hca else 16384), bits=bits,
                page=page, pad=rng.choice([0, 0, 1]) if b > 1 else 0)


def _lens(case):
    """Tokens of each sequence: the first has max_len, the others are spread below it, the last `pad` have none."""
    n = case["b"]
    out = [case["max_len"]] + [1 + int((case["max_len"] - 1) * ((i * RATIO_GOLD) % 1.0)) for i in range(1, n)]
    for i in range(n - case["pad"], n):
        out[i] = 0
    return out


def _counts(case):
    """Rows of each sequence of a write or read."""
    if not case["ragged"]:
        return [case["s"]] * case["b"]
    return [case["s"]] + [int((case["s"] + 1) * ((i * RATIO_GOLD) % 1.0)) for i in range(1, case["b"])]


def _row_bytes(d, bits):
    return d * bits // 8 + d // GROUP


def work(case):
    if case["op"] in ("write", "read"):
        n, d, e = sum(_counts(case)), case["d"], 4 if case["fp32"] else 2
        # a write is measured with the read of the same rows: x in, cache out, cache in, rows out
        return {"bytes": n * (d * e + _row_bytes(d, case["bits"])) * (2 if case["op"] == "write" else 1), "flops": n * d}
    byts = flops = 0
    for n in _lens(case):
        ts = [n - case["s_q"] + i for i in range(case["s_q"])]
        if case["op"] == "index":
            vis = [max(0, t + 1) // case["ratio"] for t in ts]
            need = [v for v in vis if v > case["topk"]]   # a row that takes every block needs no scores
            byts += (max(need) if need else 0) * _row_bytes(case["d_I"], case["bits"])
            byts += len(need) * case["H_I"] * (2 * case["d_I"] + 4) + case["s_q"] * case["topk"] * 4
            flops += sum(need) * 2 * case["H_I"] * case["d_I"]
        else:
            vis = [max(0, t + 1) // case["ratio"] for t in ts]
            sel = [min(v, case["topk"]) if case["topk"] else v for v in vis]
            win = [min(t + 1, case["window"]) if t >= 0 else 0 for t in ts]
            rows = min(max(vis), sum(sel)) + (min(max(ts) + 1, case["window"] + case["s_q"] - 1) if max(ts) >= 0 else 0)
            byts += rows * _row_bytes(case["d"], case["bits"])
            byts += case["s_q"] * (case["H"] * (4 * case["d"] + 4) + 4 * case["topk"])
            flops += 4 * case["H"] * case["d"] * (sum(sel) + sum(win))
    return {"bytes": byts, "flops": flops}


# -------------------------------------------------- the cache, plain form

def _pow2(e):
    """2^e in fp32, exactly, for whole numbers e in [-126, 127] (0 for -127)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _code_values(bits):
    """The value of every code."""
    if bits == 4:
        mags = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        return torch.tensor(mags + [-m for m in mags], device=DEV)
    vals = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = (m / 8.0) * 2.0 ** -6 if e == 0 else (1.0 + m / 8.0) * 2.0 ** (e - 7)
        vals.append(-v if c & 128 else v)
    vals[127] = vals[255] = float("nan")
    return torch.tensor(vals, device=DEV)


def _areas(cache, page, d, bits):
    """The code and scale bytes of the cache's rows, [n_pages, page, bytes], as views."""
    cb = d * bits // 8
    return cache[:, :page * cb].unflatten(1, (page, cb)), cache[:, page * cb:].unflatten(1, (page, d // GROUP))


def _encode(x, bits):
    """fp32 rows [..., d] -> (code bytes [..., d*bits/8], scale bytes [..., d/32])."""
    g = x.unflatten(-1, (-1, GROUP))
    amax = g.abs().amax(-1)
    m, ex = torch.frexp(amax)                    # amax = m 2^ex, m in [0.5, 1)
    lead, top = (0.75, 3) if bits == 4 else (0.875, 9)   # the largest code is lead * 2^top
    e = torch.where(m <= lead, ex - top, ex - top + 1).clamp_min(MIN_EXP)
    e = torch.where(amax == 0, torch.full_like(e, MIN_EXP), e)
    y = g * _pow2(-e).unsqueeze(-1)
    a = y.abs()
    sign = torch.signbit(y)
    if bits == 4:
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        r = torch.round(a / step) * step         # ties to even
        code = torch.where(r < 2, r * 2, torch.where(r < 4, r + 2, r / 2 + 4)).to(torch.uint8)
        code = (code | (sign.to(torch.uint8) << 3)).flatten(-2)
        code = code[..., 0::2] | (code[..., 1::2] << 4)
    else:
        ax = (torch.frexp(a)[1] - 1).clamp_min(-6)
        n = torch.round(a * _pow2(3 - ax)).to(torch.int32)   # a in steps of 2^(ax - 3); ties to even
        # a step count of 16 is the next exponent's 8: the sum carries into it
        code = torch.where(n < 8, n, n - 8 + ((ax + 7) << 3)) | (sign.to(torch.int32) << 7)
        code = code.to(torch.uint8).flatten(-2)
    return code, (e + 127).to(torch.uint8)


def _decode(codes, scales, values, bits, dtype=torch.float32):
    if bits == 4:
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = values.to(dtype)[codes.int()].unflatten(-1, (-1, GROUP))
    return (v * _pow2(scales.int() - 127).to(dtype).unsqueeze(-1)).flatten(-2)


def _slots(table, page, pos):
    """Flat slots (page id * page + row) of positions pos [b, ...] int64."""
    r = pos % (table.shape[1] * page)
    flat = (r // page).flatten(1)
    return table.long().gather(1, flat).view_as(r) * page + r % page


def _rows(st, cache, slots, d, dtype=torch.float32):
    page, bits = st["page"], st["bits"]
    codes, scales = _areas(cache, page, d, bits)
    p, o = slots // page, slots % page
    return _decode(codes[p, o], scales[p, o], st["values"], bits, dtype)


# ---------------------------------------------------------------- inputs

def _gen(seed, salt=0):
    return torch.Generator(device=DEV).manual_seed(seed * 1000003 + salt)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _filled(g, n_pages, page, d, bits):
    """A cache whose rows are bf16 N(0, 1) draws, quantised."""
    cache = torch.empty(n_pages, page * _row_bytes(d, bits), dtype=torch.uint8, device=DEV)
    codes, scales = _areas(cache, page, d, bits)
    step = max(1, (1 << 26) // (page * d))
    for i in range(0, n_pages, step):
        x = _randn(g, min(step, n_pages - i), page, d).bfloat16().float()
        codes[i:i + step], scales[i:i + step] = _encode(x, bits)
    return cache


def _tables(g, b, *widths):
    """Page tables of the given widths over one pool, its pages in random order."""
    total = b * sum(widths)
    ids = torch.randperm(total, generator=g, device=DEV).int()
    out, at = [], 0
    for w in widths:
        out.append(ids[at:at + b * w].view(b, w).contiguous())
        at += b * w
    return total, out


def _ints(xs):
    return torch.tensor(xs, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g, op, page, bits, b = _gen(seed), case["op"], case["page"], case["bits"], case["b"]
    st = dict(case, values=_code_values(bits))
    if op in ("write", "read"):
        s, d = case["s"], case["d"]
        dtype = torch.float32 if case["fp32"] else torch.bfloat16
        counts = _counts(case)
        pos0 = [37 * (i + 1) + (seed * 13 + 7 * i) % 29 for i in range(b)]
        width = -(-(s + max(pos0)) // page)
        n_pages, (table,) = _tables(g, b, width)
        if op == "write":
            st["x"] = _randn(g, b, s, d).to(dtype)
            st["cache"] = torch.zeros(n_pages, page * _row_bytes(d, bits), dtype=torch.uint8, device=DEV)
        else:
            st["cache"] = _filled(g, n_pages, page, d, bits)
        st.update(table=table, pos0=_ints(pos0), counts=_ints(counts), dtype=dtype,
                  out=torch.zeros(b, s, d, dtype=dtype, device=DEV),
                  pos=torch.tensor(pos0, device=DEV)[:, None] + torch.arange(s, device=DEV),
                  live=torch.arange(s, device=DEV) < torch.tensor(counts, device=DEV)[:, None])
        bi = torch.cat([torch.full((n,), i) for i, n in enumerate(counts)]).to(DEV)
        ri = torch.cat([torch.arange(n) for n in counts]).to(DEV)
        st["which"] = (bi, ri)                      # the rows that the call writes
        return st
    lens, s_q = _lens(case), case["s_q"]
    st["seq_lens"] = _ints(lens)
    n_c = max(1, max(lens) // case["ratio"])
    width = -(-n_c // page)
    st["t"] = (torch.tensor(lens, device=DEV) - s_q)[:, None] + torch.arange(s_q, device=DEV)   # positions of the queries
    if op == "index":
        H, d = case["H_I"], case["d_I"]
        n_pages, (st["table"],) = _tables(g, b, width)
        st["cache"] = _filled(g, n_pages, page, d, bits)
        st["q"] = _randn(g, b, s_q, H, d).bfloat16()
        st["w"] = _randn(g, b, s_q, H) / 2
        st["n_cap"] = n_c
        if own:
            from compressed_sparse_attention_sum_gb300 import serve
            st["ws"] = torch.empty(serve.csa_indexer_topk_decode_workspace_size(b, s_q, H, d, width * page), dtype=torch.uint8,
                                   device=DEV)
        return st
    H, d, window, topk = case["H"], case["d"], case["window"], case["topk"]
    raw_width = -(-(window + s_q - 1) // page) + 1
    n_pages, (st["raw_table"], st["cmp_table"]) = _tables(g, b, raw_width, width)
    st["cache"] = _filled(g, n_pages, page, d, bits)
    st["q"] = _randn(g, b, s_q, H, d).bfloat16()
    st["sink"] = _randn(g, H)
    st["scale"] = d ** -0.5
    st["idx"] = None
    st["n_cap"] = n_c
    if topk:
        # as the indexer writes them: min(topk, visible) distinct blocks, ascending, -1 behind; a tenth of the places -1
        vis = ((st["t"] + 1).clamp_min(0) // case["ratio"])[..., None]
        u = torch.rand(b, s_q, max(n_c, topk), generator=g, device=DEV)
        j = torch.arange(max(n_c, topk), device=DEV)
        u = torch.where(j < vis, u, u + 2)
        pick = u.topk(topk, dim=-1, largest=False).indices
        pick = torch.where(pick < vis, pick, torch.full_like(pick, 1 << 30)).sort(-1).values
        pick = torch.where(pick == 1 << 30, torch.full_like(pick, -1), pick)
        drop = torch.rand(pick.shape, generator=g, device=DEV) < 0.1
        st["idx"] = torch.where(drop, torch.full_like(pick, -1), pick).int().contiguous()
    if own:
        from compressed_sparse_attention_sum_gb300 import serve
        st["ws"] = torch.empty(serve.csa_attn_decode_workspace_size(b, s_q, H, d, window, topk if topk else width * page),
                               dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------- run

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from compressed_sparse_attention_sum_gb300 import serve
    op, page, bits = st["op"], st["page"], st["bits"]
    if op == "write":
        serve.csa_cache_write(st["x"], st["cache"], st["table"], st["pos0"], page, bits, counts=st["counts"])
    if op in ("write", "read"):
        return serve.csa_cache_read(st["cache"], st["table"], st["pos0"], st["out"], page, bits, counts=st["counts"])
    if op == "index":
        return serve.csa_indexer_topk_decode(st["q"], st["cache"], st["table"], st["w"], st["seq_lens"], st["topk"], st["ratio"],
                                             page, bits, workspace=st["ws"])
    return serve.csa_attn_decode(st["q"], st["cache"], st["raw_table"], st["cmp_table"], st["idx"], st["sink"], st["seq_lens"],
                                 st["scale"], st["ratio"], st["window"], page, bits, workspace=st["ws"])


def _run_plain(st):
    op, page, bits = st["op"], st["page"], st["bits"]
    if op in ("write", "read"):
        slots = _slots(st["table"], page, st["pos"])
        if op == "write":
            bi, ri = st["which"]
            codes, scales = _areas(st["cache"], page, st["d"], bits)
            to = slots[bi, ri]
            codes[to // page, to % page], scales[to // page, to % page] = _encode(st["x"][bi, ri].float(), bits)
        v = _rows(st, st["cache"], slots, st["d"])
        return torch.where(st["live"][..., None], v.to(st["dtype"]), st["out"])
    vis = ((st["t"] + 1).clamp_min(0) // st["ratio"])[..., None]
    if op == "index":
        # scores next to the last selected one decide: 64 bits
        b, topk, n = st["b"], st["topk"], st["n_cap"]
        j = torch.arange(n, device=DEV)
        k = _rows(st, st["cache"], _slots(st["table"], page, j.expand(b, n)), st["d_I"], torch.float64)
        s = torch.matmul(st["q"].double().flatten(1, 2), k.transpose(1, 2)).relu_().unflatten(1, (st["s_q"], st["H_I"]))
        s = (s * st["w"].double()[..., None]).sum(2)
        s = torch.where(j < vis, s, torch.full_like(s, -math.inf))
        m = min(topk, n)
        best = s.sort(dim=-1, descending=True, stable=True).indices[..., :m]      # ties: the lower block first
        best = torch.where(torch.arange(m, device=DEV) < vis, best, torch.full_like(best, n))
        best = best.sort(-1).values
        out = torch.full((b, st["s_q"], topk), -1, dtype=torch.int32, device=DEV)
        out[..., :m] = torch.where(best < n, best, torch.full_like(best, -1)).int()
        return out
    b, s_q, d = st["b"], st["s_q"], st["d"]
    t = st["t"][..., None]
    wpos = t - torch.arange(st["window"] - 1, -1, -1, device=DEV)                # [b, s_q, W]
    cpos = st["idx"].long() if st["idx"] is not None else torch.arange(st["n_cap"], device=DEV).expand(b, s_q, -1)
    ok = torch.cat((wpos >= 0, (cpos >= 0) & (cpos < vis)), -1)
    slots = torch.cat((_slots(st["raw_table"], page, wpos.clamp_min(0)), _slots(st["cmp_table"], page, cpos.clamp_min(0))), -1)
    kv = _rows(st, st["cache"], slots, d)                                              # [b, s_q, n, d]
    z = torch.matmul(st["q"].float(), kv.transpose(-1, -2)) * st["scale"]              # [b, s_q, H, n]
    z = torch.where(ok[..., None, :], z, torch.full_like(z, -math.inf))
    sink = st["sink"][:, None]
    top = torch.maximum(z.amax(-1, keepdim=True), sink)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True) + torch.exp(sink - top)
    o = torch.matmul(p, kv) / total
    return o.to(st["q"].dtype), (top + torch.log(total)).squeeze(-1)


# ----------------------------------------------------------------- exact

def _grid(bits):
    """The non-negative code values in rising order, 64 bits."""
    if bits == 4:
        return torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    small = [i * 2.0 ** -9 for i in range(8)]
    rest = [(8 + i) * 2.0 ** (e - 10) for e in range(1, 16) for i in range(8)]
    return torch.tensor((small + rest)[:127], dtype=torch.float64, device=DEV)


def _nearest(x, bits):
    """Rows [n, d] as the cache holds them: the nearest grid value times the group's power of two."""
    grid, top = _grid(bits), TOP[bits]
    g = x.double().reshape(x.shape[0], -1, GROUP)
    most = g.abs().amax(-1, keepdim=True)
    unit = torch.full_like(most, 2.0 ** MIN_EXP)
    guess = torch.exp2(torch.floor(torch.log2(torch.where(most > 0, most, torch.ones_like(most)) / top)))
    for k in (2.0, 1.0, 0.5):                     # the smallest power of two that holds the group
        cand = guess * k
        fits = (cand * top >= most) & (most > 0) & (cand > 2.0 ** MIN_EXP)
        unit = torch.where(fits, cand, unit)
    a = (g / unit).abs()
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, len(grid) - 1)
    below, above = a - grid[hi - 1], grid[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    v = torch.where(up, grid[hi], grid[hi - 1])
    return (torch.sign(g) * v * unit).reshape(x.shape)


def _held(st, table, i, pos):
    """Rows of sequence i at positions pos from the cache's bytes, 64 bits."""
    page, bits = st["page"], st["bits"]
    d = st["d_I"] if st["op"] == "index" else st["d"]
    slot = pos % (table.shape[1] * page)
    at = table[i].long()[slot // page] * (page * _row_bytes(d, bits))
    row = slot % page
    cb, n_g = d * bits // 8, d // GROUP
    flat = st["cache"].view(-1)
    codes = flat[(at + row * cb)[:, None] + torch.arange(cb, device=DEV)].long()
    scale = flat[(at + page * cb + row * n_g)[:, None] + torch.arange(n_g, device=DEV)].double()
    if bits == 4:
        codes = torch.stack([(codes >> s) & 15 for s in (0, 4)], 2).reshape(len(pos), d)
        mag, neg = codes & 7, codes >> 3
    else:
        mag, neg = codes & 127, codes >> 7
    v = _grid(bits)[mag] * (1 - 2 * neg)
    return v * torch.exp2(scale - 127).repeat_interleave(GROUP, 1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("write", "read"):
        out = torch.zeros(case["b"], case["s"], case["d"], dtype=torch.float64, device=DEV)
        for i, n in enumerate(_counts(case)):
            if n:
                out[i, :n] = (_nearest(st["x"][i, :n], case["bits"]) if case["op"] == "write"
                              else _held(st, st["table"], i, st["pos"][i, :n]))
        return out
    if case["op"] == "index":
        out = torch.full((case["b"], case["s_q"], case["topk"]), -1, dtype=torch.int32, device=DEV)
        for i, n in enumerate(_lens(case)):
            last = max(0, n) // case["ratio"]
            k = _held(st, st["table"], i, torch.arange(last, device=DEV))
            for r in range(case["s_q"]):
                vis = max(0, n - case["s_q"] + r + 1) // case["ratio"]
                dots = k[:vis] @ st["q"][i, r].double().T
                score = (dots.clamp(min=0) @ st["w"][i, r].double())
                order = torch.argsort(score, descending=True, stable=True)[:case["topk"]]
                out[i, r, :len(order)] = order.sort().values.int()
        return out
    o = torch.zeros(case["b"], case["s_q"], case["H"], case["d"], dtype=torch.float64, device=DEV)
    lse = torch.empty(case["b"], case["s_q"], case["H"], dtype=torch.float64, device=DEV)
    sink = st["sink"].double()
    for i, n in enumerate(_lens(case)):
        for r in range(case["s_q"]):
            t = n - case["s_q"] + r
            vis = max(0, t + 1) // case["ratio"]
            js = st["idx"][i, r].long() if st["idx"] is not None else torch.arange(vis, device=DEV)
            js = js[(js >= 0) & (js < vis)]
            ws = torch.arange(max(0, t - case["window"] + 1), t + 1, device=DEV)
            kv = torch.cat([_held(st, st["raw_table"], i, ws), _held(st, st["cmp_table"], i, js)])
            z = torch.cat([st["q"][i, r].double() @ kv.T * st["scale"], sink[:, None]], 1)
            lse[i, r] = torch.logsumexp(z, 1)
            o[i, r] = torch.exp(z[:, :-1] - lse[i, r][:, None]) @ kv
    return o, lse
