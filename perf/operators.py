"""The serving operators around the sparse indexer, as measured workloads.

Four operators make up one attention layer's part of a serving step:

  plan      block tables, slot maps and positions built from request lengths;
  table     rotary cosine/sine tables, also scaled for long contexts;
  norm      per-head RMS norm of queries and keys, rotary turn and cache insert
            in one pass;
  attend    attention of the new tokens over the paged key-value cache, over the
            whole context or over the positions the indexer selected.

`run` computes each either in a plain form (elementary torch operations in 32
bits, 64 for angles) or, with `own` set, through the package's entry points.
`exact` gives the same outputs in 64 bits, written apart from the plain form.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "e4m3": 1}
E4M3_MAX = 448.0
EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step of a busy server: every request adds one token, one in
        # 64 of them opens a new page
        {"name": "plan-decode", "op": "plan", "B": 256, "max_blocks": 512, "page": 64,
         "cached_lo": 1024, "cached_hi": 32000, "new_lo": 1, "new_hi": 1, "pad": 0},
        # a mixed step: chunked prefills of very different lengths beside
        # requests that sit the step out, token arrays padded to a fixed size
        {"name": "plan-mixed", "op": "plan", "B": 129, "max_blocks": 2048, "page": 16,
         "cached_lo": 0, "cached_hi": 20000, "new_lo": 0, "new_hi": 1000, "pad": 777},
        # the table of a short-context layer, half of a 128-wide head turned
        {"name": "table-4k", "op": "table", "num_pos": 4096, "rot": 64, "pos0": 0,
         "scaling": "none", "factor": 1.0, "orig": 0},
        # a long-context table: frequencies blended by wavelength
        {"name": "table-256k-yarn", "op": "table", "num_pos": 262144, "rot": 128, "pos0": 0,
         "scaling": "yarn", "factor": 8.0, "orig": 32768},
        # the new tokens of a decode batch, sliced out of a fused projection
        {"name": "norm-decode", "op": "norm", "N": 64, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "interleaved": False, "norm": True, "dtype": "bf16", "cache": "bf16", "page": 64,
         "num_pos": 32768, "pad": 0},
        # a long prefill, interleaved pairs over half of each head
        {"name": "norm-prefill", "op": "norm", "N": 32768, "Hq": 32, "Hkv": 8, "D": 128,
         "rot": 64, "interleaved": True, "norm": True, "dtype": "bf16", "cache": "bf16",
         "page": 64, "num_pos": 32768, "pad": 0},
        # an odd chunk into an 8-bit cache, with padding rows
        {"name": "norm-chunk-e4m3", "op": "norm", "N": 1037, "Hq": 24, "Hkv": 4, "D": 256,
         "rot": 64, "interleaved": False, "norm": True, "dtype": "fp16", "cache": "e4m3",
         "page": 16, "num_pos": 8192, "pad": 5},
        # one request at the start of its answer: latency alone
        {"name": "attend-one", "op": "attend", "B": 1, "lo": 129, "hi": 129, "next_n": 1,
         "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "cache": "bf16", "page": 64,
         "order": "hnd", "k": 0, "window": 0, "softcap": 0.0, "empty": False},
        # the batched decode's contexts over the whole cache
        {"name": "attend-batch", "op": "attend", "B": 64, "lo": 8192, "hi": 32768, "next_n": 1,
         "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "cache": "bf16", "page": 64,
         "order": "hnd", "k": 0, "window": 0, "softcap": 0.0, "empty": False},
        # two long requests with a speculated token each, 8-bit cache: few rows,
        # so the work lies along the cache's length
        {"name": "attend-long-e4m3", "op": "attend", "B": 2, "lo": 131072, "hi": 131072,
         "next_n": 2, "Hq": 64, "Hkv": 8, "D": 128, "dtype": "bf16", "cache": "e4m3",
         "page": 64, "order": "hnd", "k": 0, "window": 0, "softcap": 0.0, "empty": False},
        # the batched decode over the indexer's 2048 positions per row
        {"name": "attend-topk", "op": "attend", "B": 64, "lo": 4096, "hi": 16384, "next_n": 1,
         "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "cache": "bf16", "page": 64,
         "order": "nhd", "k": 2048, "window": 0, "softcap": 0.0, "empty": False},
        # ragged short requests, one of them empty, capped scores, a sliding
        # window, a group of five heads, 64-wide heads, 16-token pages
        {"name": "attend-ragged-cap", "op": "attend", "B": 37, "lo": 1, "hi": 5000,
         "next_n": 2, "Hq": 20, "Hkv": 4, "D": 64, "dtype": "fp16", "cache": "fp16",
         "page": 16, "order": "nhd", "k": 0, "window": 1500, "softcap": 30.0, "empty": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "table", "norm", "norm", "attend", "attend", "attend"])
    if op == "plan":
        decode = rng.random() < 0.4
        B = _log_int(rng, 1, 600)
        page = rng.choice([16, 32, 64, 128])
        cached_hi = _log_int(rng, 1, 24000)
        new_hi = 1 if decode else _log_int(rng, 2, max(2, 120000 // B))
        return {"op": "plan", "B": B, "max_blocks": -(-(cached_hi + new_hi) // page) + rng.randint(0, 9),
                "page": page, "cached_lo": 0, "cached_hi": cached_hi,
                "new_lo": 1 if decode else 0, "new_hi": new_hi, "pad": rng.randint(0, 300)}
    if op == "table":
        rot = 2 * rng.randint(2, 64)
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return {"op": "table", "num_pos": _log_int(rng, 1, 200000), "rot": rot,
                "pos0": rng.choice([0, 0, rng.randint(1, 1000000)]), "scaling": scaling,
                "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 10.0, 32.0]),
                "orig": rng.choice([4096, 8192, 32768]) if scaling == "yarn" else 0}
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "fp16"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    if op == "norm":
        interleaved = rng.random() < 0.5
        N = _log_int(rng, 1, 20000 if cache != "e4m3" else 3_000_000 // (Hkv * D))
        return {"op": "norm", "N": N, "Hq": Hkv * rng.randint(1, 8), "Hkv": Hkv, "D": D,
                "rot": 2 * rng.randint(0, D // 2) if interleaved else 16 * rng.randint(0, D // 16),
                "interleaved": interleaved, "norm": rng.random() < 0.8, "dtype": dtype,
                "cache": cache, "page": page, "num_pos": _log_int(rng, 16, 65536),
                "pad": rng.choice([0, 0, 1, 7]) if N > 8 else 0}
    sparse = rng.random() < 0.4
    hi = _log_int(rng, 1, 100000)
    most = 1_500_000_000 // (Hkv * D * 2 * BYTES[cache] * hi)
    B = _log_int(rng, 1, max(1, min(200, most)))
    # a drawn list of positions is an argsort over all positions: keep it small
    if sparse:
        hi = min(hi, max(1, 2_000_000 // B))
    next_n = rng.choice([1, 1, 2, 3])
    return {"op": "attend", "B": B, "lo": next_n if rng.random() < 0.7 else max(next_n, hi),
            "hi": max(next_n, hi), "next_n": next_n,
            "Hq": Hkv * rng.choice([1, 2, 4, 5, 8, 12, 16]), "Hkv": Hkv, "D": D, "dtype": dtype,
            "cache": cache, "page": page, "order": rng.choice(["hnd", "nhd"]),
            "k": _log_int(rng, 1, 2048) if sparse else 0,
            "window": 0 if sparse else rng.choice([0, 0, 0, _log_int(rng, 1, 4000)]),
            "softcap": rng.choice([0.0, 0.0, 0.0, 20.0]),
            "empty": B > 1 and rng.random() < 0.3}


# ------------------------------------------------------------------ inputs

def _case_rng(case):
    # lengths belong to the case, not to the seed: the work is the same for every seed
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _plan_lens(case):
    r = _case_rng(case)
    cached = [r.randint(case["cached_lo"], case["cached_hi"]) for _ in range(case["B"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return cached, new


def _attend_lens(case):
    r = _case_rng(case)
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    lens[-1] = case["hi"]
    if case["empty"]:
        lens[0] = 0
    return lens


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_plan(case, g):
    cached, new = _plan_lens(case)
    B, page, mb = case["B"], case["page"], case["max_blocks"]
    have = [-(-c // page) for c in cached]
    need = sum(max(0, -(-(c + n) // page) - h) for c, n, h in zip(cached, new, have))
    used = sum(have)
    num_blocks = used + need + 1 + (used + need) // 4
    perm = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    cols = torch.arange(mb, device="cuda")
    live = cols[None, :] < torch.tensor(have, device="cuda")[:, None]
    bt = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
    bt[live] = perm[:used]
    return {"cached": _i32(cached), "new": _i32(new), "bt": bt,
            "free": perm[used:].contiguous(), "head": _i32([0]),
            "num_tokens": sum(new) + case["pad"], "num_blocks": num_blocks, "page": page}


def _paged(values, order):
    """[blocks, Hkv, page, D] values as the cache holds them: `hnd` keeps a
    head's page contiguous, `nhd` a token's heads (a strided view)."""
    if order == "hnd":
        return values
    return values.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)


def _randn(shape, dtype, g):
    if dtype == torch.float8_e4m3fn:
        out = torch.empty(shape, dtype=dtype, device="cuda")
        for i in range(0, shape[0], 4096):
            part = (min(4096, shape[0] - i),) + tuple(shape[1:])
            out[i:i + 4096] = torch.randn(part, dtype=torch.float16, device="cuda",
                                          generator=g).to(dtype)
        return out
    return torch.randn(shape, dtype=dtype, device="cuda", generator=g)


def _prepare_norm(case, g):
    N, Hq, Hkv, D, page = (case[x] for x in ("N", "Hq", "Hkv", "D", "page"))
    dt, ct = DTYPES[case["dtype"]], DTYPES[case["cache"]]
    # q, k and v are slices of one projection's output, as a layer has them
    qkv = torch.randn(N, Hq + 2 * Hkv, D, dtype=dt, device="cuda", generator=g)
    num_blocks = -(-N // page) + N // (4 * page) + 1
    slots = torch.randperm(num_blocks * page, generator=g, device="cuda")[:N].contiguous()
    if case["pad"]:
        slots[torch.randperm(N, generator=g, device="cuda")[:case["pad"]]] = -1
    half = case["rot"] // 2
    ang = (torch.arange(case["num_pos"], dtype=torch.float64, device="cuda")[:, None]
           * BASE ** (-torch.arange(half, dtype=torch.float64, device="cuda") / max(half, 1)))
    s = {"q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hkv], "v": qkv[:, Hq + Hkv:],
         "positions": torch.randint(0, case["num_pos"], (N,), generator=g, device="cuda",
                                    dtype=torch.int32),
         "cos": torch.cos(ang).float(), "sin": torch.sin(ang).float(), "rot": case["rot"],
         "interleaved": case["interleaved"], "slots": slots, "qw": None, "kw": None,
         "k_scale": None, "v_scale": None,
         "k_cache": torch.zeros(num_blocks, Hkv, page, D, device="cuda").to(ct),
         "v_cache": torch.zeros(num_blocks, Hkv, page, D, device="cuda").to(ct)}
    if case["norm"]:
        s["qw"] = 1 + 0.2 * torch.randn(D, device="cuda", generator=g)
        s["kw"] = 1 + 0.2 * torch.randn(D, device="cuda", generator=g)
    if case["cache"] == "e4m3":
        s["k_scale"] = 0.01 + 0.02 * torch.rand(Hkv, device="cuda", generator=g)
        s["v_scale"] = 0.01 + 0.02 * torch.rand(Hkv, device="cuda", generator=g)
    return s


def _prepare_attend(case, g):
    lens = _attend_lens(case)
    B, n, Hq, Hkv, D, page = (case[x] for x in ("B", "next_n", "Hq", "Hkv", "D", "page"))
    have = [-(-x // page) for x in lens]
    mb, used = max(max(have), 1), sum(have)
    num_blocks = used + used // 4 + 1
    perm = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    live = torch.arange(mb, device="cuda")[None, :] < torch.tensor(have, device="cuda")[:, None]
    bt = torch.zeros((B, mb), dtype=torch.int32, device="cuda")
    bt[live] = perm[:used]
    ct, shape = DTYPES[case["cache"]], (num_blocks, Hkv, page, D)
    s = {"q": 2 * torch.randn(B * n, Hq, D, dtype=DTYPES[case["dtype"]], device="cuda",
                              generator=g),
         "k_cache": _paged(_randn(shape, ct, g), case["order"]),
         "v_cache": _paged(_randn(shape, ct, g), case["order"]),
         "bt": bt, "lens": _i32(lens), "next_n": n, "scale": D ** -0.5,
         "softcap": case["softcap"], "window": case["window"], "topk": None,
         "k_scale": None, "v_scale": None}
    if case["cache"] == "e4m3":
        s["k_scale"] = 0.5 + torch.rand(Hkv, device="cuda", generator=g)
        s["v_scale"] = 0.5 + torch.rand(Hkv, device="cuda", generator=g)
    if case["k"]:
        # distinct positions of the row's window in random order, -1 after the
        # last, as the indexer's selection leaves them
        ends = _row_ends(s["lens"], n)
        order = torch.rand(B * n, max(max(lens), 1), device="cuda", generator=g)
        order[torch.arange(order.shape[1], device="cuda")[None, :] >= ends[:, None]] = 2.0
        pick = torch.full((B * n, case["k"]), -1, dtype=torch.int32, device="cuda")
        m = min(case["k"], order.shape[1])
        at = order.argsort(dim=1)[:, :m].to(torch.int32)
        pick[:, :m] = torch.where(torch.arange(m, device="cuda")[None, :] < ends[:, None], at,
                                  pick[:, :m])
        s["topk"] = pick
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    if case["op"] == "table":
        # what a program holds here is a configuration; the seed moves the
        # first position, as a table that is extended does
        s = {x: case[x] for x in ("num_pos", "rot", "scaling", "factor", "orig")}
        s["pos0"] = case["pos0"] + int(seed) % 4096
    elif case["op"] == "plan":
        s = _prepare_plan(case, g)
    elif case["op"] == "norm":
        s = _prepare_norm(case, g)
    else:
        s = _prepare_attend(case, g)
    s["op"] = case["op"]
    return s


def _row_ends(lens, next_n):
    """Window length of every row: row (b, j) sees [0, L_b - next_n + j]."""
    j = torch.arange(next_n, device=lens.device)
    return (lens.long()[:, None] - next_n + 1 + j[None, :]).clamp(min=0).reshape(-1)


# ------------------------------------------------------------------ plain forms

def _plain_plan(s):
    page, bt, N = s["page"], s["bt"], s["num_tokens"]
    cached, new = s["cached"].long(), s["new"].long()
    ctx = cached + new
    have = (cached + page - 1) // page
    take = ((ctx + page - 1) // page - have).clamp(min=0)
    start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    pstart = torch.cat([take.new_zeros(1), take.cumsum(0)])
    col = torch.arange(bt.shape[1], device=bt.device)[None, :] - have[:, None]
    fresh = (col >= 0) & (col < take[:, None])
    at = (s["head"].long() + pstart[:-1, None] + col).clamp(0, s["free"].numel() - 1)
    bt.copy_(torch.where(fresh, s["free"][at], bt))
    t = torch.arange(N, device=bt.device)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=new.numel() - 1)
    live = t < start[-1]
    pos = torch.where(live, cached[b] + t - start[b], 0)
    page_id = bt[b, (pos // page).clamp(max=bt.shape[1] - 1)].long()
    slots = torch.where(live, page_id * page + pos % page, -1)
    return {"context_lens": ctx.int(), "query_start": start.int(), "slot_mapping": slots,
            "positions": pos.int(), "token_seq": torch.where(live, b, -1).int(),
            "pool_head": s["head"] + pstart[-1:].int(), "block_table": bt}


def _plain_freqs(s):
    rot, base, factor = s["rot"], BASE, s["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    if s["scaling"] == "ntk":
        base = BASE * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if s["scaling"] == "linear":
        f = f / factor
    if s["scaling"] == "yarn":
        dims = [rot * math.log(s["orig"] / (turns * 2 * math.pi)) / (2 * math.log(BASE))
                for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(dims[0]), 0), min(math.ceil(dims[1]), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
    return f


def _mscale(s):
    return 0.1 * math.log(s["factor"]) + 1.0 if s["scaling"] == "yarn" else 1.0


def _plain_table(s):
    pos = torch.arange(s["num_pos"], dtype=torch.float64, device="cuda") + s["pos0"]
    ang = pos[:, None] * _plain_freqs(s)[None, :]
    return {"cos": (torch.cos(ang) * _mscale(s)).float(), "sin": (torch.sin(ang) * _mscale(s)).float()}


def _plain_turn(x, c, sn, rot, interleaved):
    half = rot // 2
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :half], x[..., half:rot])
    c, sn = c[:, None, :], sn[:, None, :]
    u, w = a * c - b * sn, a * sn + b * c
    turned = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_normed(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _plain_store(cache, slots, x, scale):
    page = cache.shape[2]
    if scale is not None:
        x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    keep = slots >= 0
    at = slots[keep]
    rows = x[keep].to(cache.dtype)
    raw, vals = (cache, rows) if cache.dtype != torch.float8_e4m3fn else (
        cache.view(torch.uint8), rows.view(torch.uint8))
    raw[at // page, :, at % page] = vals


def _plain_norm(s):
    pos = s["positions"].long()
    c, sn = s["cos"][pos], s["sin"][pos]
    q = _plain_turn(_plain_normed(s["q"], s["qw"]), c, sn, s["rot"], s["interleaved"])
    k = _plain_turn(_plain_normed(s["k"], s["kw"]), c, sn, s["rot"], s["interleaved"])
    _plain_store(s["k_cache"], s["slots"], k, s["k_scale"])
    _plain_store(s["v_cache"], s["slots"], s["v"].float(), s["v_scale"])
    return {"q": q.to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_softmax(x, seen, softcap):
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == -math.inf, 0.0))
    l = p.sum(-1, keepdim=True)
    return p, l, (m + torch.log(l)).squeeze(-1)


def _plain_pages(cache, at, scale):
    x = cache[at] if cache.dtype != torch.float8_e4m3fn else (
        cache.view(torch.uint8)[at].view(cache.dtype))
    x = x.float()
    return x if scale is None else x * scale[:, None, None]


def _plain_attend(s):
    n, (R, Hq, D) = s["next_n"], s["q"].shape
    B, Hkv, page = R // n, s["k_cache"].shape[1], s["k_cache"].shape[2]
    ends = _row_ends(s["lens"], n)
    q = s["q"].float() * s["scale"]
    if s["topk"] is None:
        bt = s["bt"].long()
        k = _plain_pages(s["k_cache"], bt, s["k_scale"]).transpose(1, 2).reshape(B, Hkv, -1, D)
        v = _plain_pages(s["v_cache"], bt, s["v_scale"]).transpose(1, 2).reshape(B, Hkv, -1, D)
        q = q.view(B, n, Hkv, -1, D).transpose(1, 2).reshape(B, Hkv, -1, D)
        x = q @ k.transpose(-1, -2)
        at = torch.arange(k.shape[2], device=q.device)
        e = ends.view(B, 1, n, 1, 1)
        seen = at < e
        if s["window"]:
            seen = seen & (at >= e - s["window"])
        p, l, lse = _plain_softmax(x.view(B, Hkv, n, -1, at.numel()), seen, s["softcap"])
        o = (p.flatten(2, 3) @ v).view(B, Hkv, n, -1, D) / l.clamp(min=1e-30)
        o, lse = o.transpose(1, 2).reshape(R, Hq, D), lse.transpose(1, 2).reshape(R, Hq)
    else:
        at = s["topk"].long()
        seen = (at >= 0)[:, None, None, :]
        at = at.clamp(min=0)
        row = torch.arange(R, device=at.device)[:, None] // n
        pages, offs = s["bt"][row, at // page].long(), at % page

        def rows_of(cache, scale):
            x = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
            x = x[pages, :, offs].view(cache.dtype).float()
            return (x if scale is None else x * scale[:, None]).transpose(1, 2)

        x = q.view(R, Hkv, -1, D) @ rows_of(s["k_cache"], s["k_scale"]).transpose(-1, -2)
        p, l, lse = _plain_softmax(x, seen, s["softcap"])
        o = (p @ rows_of(s["v_cache"], s["v_scale"])) / l.clamp(min=1e-30)
        o, lse = o.reshape(R, Hq, D), lse.reshape(R, Hq)
    return {"out": o.to(s["q"].dtype), "lse": lse}


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        from sparse_attention_indexer_quant_gb300 import binding as idx
        if s["op"] == "plan":
            p = idx.plan_step(s["cached"], s["new"], s["bt"], s["free"], s["head"],
                              s["num_tokens"], s["num_blocks"], page_size=s["page"])
            return {"context_lens": p.context_lens, "query_start": p.query_start,
                    "slot_mapping": p.slot_mapping, "positions": p.positions,
                    "token_seq": p.token_seq, "pool_head": p.pool_head, "block_table": s["bt"]}
        if s["op"] == "table":
            cos, sin = idx.rope_table(s["num_pos"], s["rot"], base=BASE, scaling=s["scaling"],
                                      factor=s["factor"], orig_len=s["orig"], pos0=s["pos0"])
            return {"cos": cos, "sin": sin}
        if s["op"] == "norm":
            q = idx.qk_norm_rope_insert(
                s["q"], s["k"], s["v"], s["qw"], s["kw"], EPS, s["positions"], s["cos"],
                s["sin"], s["rot"], s["slots"], s["k_cache"], s["v_cache"],
                interleaved=s["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        out, lse = idx.paged_attention(
            s["q"], s["k_cache"], s["v_cache"], s["bt"], s["lens"], s["next_n"],
            scale=s["scale"], softcap=s["softcap"], window=s["window"], topk=s["topk"],
            k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=True)
        return {"out": out, "lse": lse}
    return {"plan": _plain_plan, "table": _plain_table, "norm": _plain_norm,
            "attend": _plain_attend}[s["op"]](s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "plan":
        cached, new = _plan_lens(case)
        page, N = case["page"], sum(new) + case["pad"]
        fresh = sum(max(0, -(-(c + n) // page) + (-c // page)) for c, n in zip(cached, new))
        partly = sum(1 for c, n in zip(cached, new) if n and c % page)
        # lengths in and out, starts; per token slot, position and request; new
        # pages read from the list and written; the partly filled page's entry
        return {"bytes": 16 * case["B"] + 12 + 16 * N + 8 * fresh + 4 * partly, "flops": 0}
    if case["op"] == "table":
        values = case["num_pos"] * case["rot"]
        return {"bytes": 4 * values, "flops": 10 * values}
    if case["op"] == "norm":
        N, Hq, Hkv, D, e = case["N"], case["Hq"], case["Hkv"], case["D"], BYTES[case["dtype"]]
        rows = min(N, case["num_pos"])
        moved = N * (2 * Hq + 2 * Hkv) * D * e + (N - case["pad"]) * 2 * Hkv * D * BYTES[case["cache"]]
        return {"bytes": moved + 12 * N + 4 * rows * case["rot"] + (8 * D if case["norm"] else 0),
                "flops": N * (Hq + Hkv) * (4 * D * case["norm"] + 3 * case["rot"])}
    n, Hq, Hkv, D = case["next_n"], case["Hq"], case["Hkv"], case["D"]
    lens = _attend_lens(case)
    keys = pairs = pages = 0
    for L in lens:
        ends = [max(0, L - n + 1 + j) for j in range(n)]
        if case["k"]:
            seen = [min(case["k"], e) for e in ends]
            # rows of one request select apart from each other
            keys += min(sum(seen), L)
            pages += min(sum(seen), -(-L // case["page"]))
        else:
            w = case["window"] or L
            seen = [min(w, e) for e in ends]
            first = max(0, ends[0] - w)
            keys += max(0, L - first)
            pages += -(-L // case["page"]) - first // case["page"]
        pairs += sum(seen)
    R = case["B"] * n
    rows = R * Hq * (2 * D * BYTES[case["dtype"]] + 4)
    return {"bytes": keys * Hkv * D * 2 * BYTES[case["cache"]] + rows + 4 * pages + 4 * case["B"]
            + 4 * R * case["k"], "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_table(s):
    """Angles as whole turns and a remainder, the frequencies from Python floats."""
    rot, f = s["rot"], []
    base = BASE * s["factor"] ** (rot / (rot - 2)) if s["scaling"] == "ntk" else BASE
    for i in range(rot // 2):
        w = math.exp(-math.log(base) * 2 * i / rot)
        if s["scaling"] == "linear":
            w /= s["factor"]
        elif s["scaling"] == "yarn":
            # dimension at which a frequency makes `turns` turns over the original length
            at = [0.5 * rot * math.log(s["orig"] / (2 * math.pi * t)) / math.log(BASE)
                  for t in (32.0, 1.0)]
            lo, hi = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
            mix = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = w / s["factor"] * mix + w * (1 - mix)
        f.append(w)
    f = torch.tensor(f, dtype=torch.float64, device="cuda")
    pos = torch.arange(s["pos0"], s["pos0"] + s["num_pos"], device="cuda").double()
    z = torch.polar(torch.tensor(_mscale(s), dtype=torch.float64, device="cuda"),
                    torch.outer(pos, f))
    return {"cos": z.real.contiguous(), "sin": z.imag.contiguous()}


def _exact_norm(s):
    pos, rot, half = s["positions"].long(), s["rot"], s["rot"] // 2
    z = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None, :]

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
        x = x.clone()
        even = torch.arange(half, device=x.device)
        a, b = (2 * even, 2 * even + 1) if s["interleaved"] else (even, even + half)
        y = torch.complex(x[..., a], x[..., b]) * z
        x[..., a], x[..., b] = y.real, y.imag
        return x

    def stored(cache, x, scale):
        out = torch.zeros(cache.shape, dtype=torch.float64, device="cuda")
        page = cache.shape[2]
        if scale is not None:  # the value that the 8-bit code is nearest to
            x = (x / scale.double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        for i, at in enumerate(s["slots"].tolist()):
            if at >= 0:
                out[at // page, :, at % page] = x[i]
        return out

    return {"q": turned(s["q"], s["qw"]),
            "k_cache": stored(s["k_cache"], turned(s["k"], s["kw"]), s["k_scale"]),
            "v_cache": stored(s["v_cache"], s["v"].double(), s["v_scale"])}


def _exact_attend(s):
    n, (R, Hq, D) = s["next_n"], s["q"].shape
    Hkv, page, lens = s["k_cache"].shape[1], s["k_cache"].shape[2], s["lens"].tolist()
    out = torch.zeros(R, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64, device="cuda")

    def rows_of(cache, scale, pages, offs):
        raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
        x = raw[pages, :, offs].view(cache.dtype).double()
        return x if scale is None else x * scale.double()[None, :, None]

    for r in range(R):
        b, end = r // n, max(0, lens[r // n] - n + 1 + r % n)
        if s["topk"] is not None:
            at = s["topk"][r].long()
            at = at[at >= 0]
        else:
            at = torch.arange(max(0, end - s["window"]) if s["window"] else 0, end, device="cuda")
        if at.numel() == 0:
            continue
        pages, offs = s["bt"][b].long()[at // page], at % page
        k = rows_of(s["k_cache"], s["k_scale"], pages, offs)
        v = rows_of(s["v_cache"], s["v_scale"], pages, offs)
        q = s["q"][r].double().view(Hkv, Hq // Hkv, D)
        x = torch.einsum("hgd,lhd->hgl", q, k) * s["scale"]
        if s["softcap"]:
            x = s["softcap"] * torch.tanh(x / s["softcap"])
        total = torch.logsumexp(x, -1)
        out[r] = torch.einsum("hgl,lhd->hgd", torch.exp(x - total[..., None]), v).reshape(Hq, D)
        lse[r] = total.reshape(Hq)
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    return {"table": _exact_table, "norm": _exact_norm, "attend": _exact_attend}[case["op"]](s)
