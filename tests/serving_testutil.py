"""Plain 64-bit forms of the serving operators (step plan, rotary tables, q/k
norm + rotary + cache insert, paged attention) and the tolerances that their
kernels are held to.

Tolerances count roundings: one to an output type t is off by at most
eps(t) / 2 relative to the value; fp32 arithmetic by 2^-24 per operation."""
import math

import numpy as np
import torch

U = 2.0 ** -24  # half a step of fp32
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E4M3_MAX = 448.0


# ------------------------------------------------------------------ step plan

def ref_plan(cached, new, block_table, free, head, num_tokens, num_blocks, page):
    """Request by request and token by token.  Returns (context_lens,
    query_start, slots, positions, token_seq, head, block_table, bad)."""
    B, max_blocks = block_table.shape
    bt = block_table.copy()
    slots = np.full(num_tokens, -1, np.int64)
    positions = np.zeros(num_tokens, np.int32)
    seqs = np.full(num_tokens, -1, np.int32)
    ctx, start, bad, t = [], [0], 0, 0
    if not 0 <= head <= len(free):
        head = len(free)
    given = head
    for b in range(B):
        c, n = int(cached[b]), int(new[b])
        if c < 0 or n < 0:
            bad, c, n = bad + 1, 0, 0
        if c + n > 2**31 - 1:
            bad, n = bad + 1, 0
        want, have = -(-(c + n) // page), -(-c // page)
        if want > max_blocks:
            bad += 1
        for i in range(have, min(want, max_blocks)):
            page_id = int(free[given]) if given < len(free) else -1
            if not 0 <= page_id < num_blocks:
                page_id, bad = -1, bad + 1
            bt[b, i] = page_id
            given += 1
        for p in range(c, c + n):
            if t < num_tokens:
                i = p // page
                page_id = int(bt[b, i]) if i < max_blocks else -1
                if i < min(have, max_blocks) and not 0 <= page_id < num_blocks:
                    page_id, bad = -1, bad + 1
                slots[t] = page_id * page + p % page if page_id >= 0 else -1
                positions[t], seqs[t] = p, b
            else:
                bad += 1
            t += 1
        ctx.append(c + n)
        start.append(t)
    return (np.array(ctx, np.int32), np.array(start, np.int32), slots, positions, seqs,
            min(given, len(free)), bt, bad)


# ------------------------------------------------------------------ rotary tables

def ref_freqs(rot, base=10000.0, scaling=None, factor=1.0, orig_len=0, beta_fast=32.0,
              beta_slow=1.0):
    """w_i in extended precision."""
    ld = np.longdouble
    i = np.arange(rot // 2).astype(ld)
    b = ld(base) * ld(factor) ** (ld(rot) / (rot - 2)) if scaling == "ntk" else ld(base)
    w = b ** (-2 * i / rot)
    if scaling == "linear":
        w = w / ld(factor)
    if scaling == "yarn":
        def dim(beta):
            return rot * math.log(orig_len / (beta * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(dim(beta_fast)), 0)
        hi = min(math.ceil(dim(beta_slow)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, ld(0.001)), 0, 1)
        w = w * (1 - ramp) + w / ld(factor) * ramp
    return w


def ref_table(pos0, num_pos, rot, mscale=1.0, **kw):
    turns = ref_freqs(rot, **kw) / (2 * np.pi)
    ang = (np.arange(pos0, pos0 + num_pos).astype(np.longdouble)[:, None] * turns[None, :])
    ang = (ang - np.floor(ang)).astype(np.float64) * (2 * np.pi)
    return mscale * np.cos(ang), mscale * np.sin(ang)


# ------------------------------------------------------------------ norm, turn, insert

def ref_turned(x, weight, eps, cos, sin, rot, interleaved):
    """x [N, H, D] float64 -> (value, sum of the magnitudes that enter it)."""
    x = x.copy()
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    half = rot // 2
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cos[:, None, :], sin[:, None, :]
    y, mag = x.copy(), np.abs(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    mag[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
    mag[..., b] = np.abs(x[..., a] * s) + np.abs(x[..., b] * c)
    return y, mag


def turned_tol(ref, mag, dim, normed, half_step, floor):
    """fp32 steps: the sum of dim squares, rsqrt (2 ulp), two products, the
    turn's two products and sum; then the rounding to the output type, whose
    smallest step is `floor`."""
    steps = (dim + 8 if normed else 0) + 4
    err = steps * U * mag
    return half_step * (np.abs(ref) + err) + err + floor


# ------------------------------------------------------------------ attention

def ref_attention(q, k, v, bt, lens, next_n, scale, softcap=0.0, window=0, topk=None):
    """q [R, Hq, D], k/v [blocks, Hkv, page, D] float64 arrays.  Row by row.
    Returns out, lse, and per (row, head) the largest |score| sum and per output
    the sum of p |v|."""
    R, Hq, D = q.shape
    Hkv, page = k.shape[1], k.shape[2]
    cap = bt.shape[1] * page
    out = np.zeros((R, Hq, D))
    lse = np.full((R, Hq), -np.inf)
    smag = np.zeros((R, Hq))
    omag = np.zeros((R, Hq, D))
    count = np.zeros(R, np.int64)
    for r in range(R):
        b = r // next_n
        L = min(max(int(lens[b]), 0), cap)
        end = max(0, L - next_n + 1 + r % next_n)
        if topk is not None:
            at = np.array([p for p in topk[r] if 0 <= p < end], np.int64)
        else:
            at = np.arange(max(0, end - window) if window else 0, end)
        pages = bt[b][at // page] if len(at) else np.zeros(0, np.int64)
        ok = (pages >= 0) & (pages < k.shape[0])
        at, pages = at[ok], pages[ok]
        count[r] = len(at)
        if not len(at):
            continue
        kk = k[pages, :, at % page]  # [n, Hkv, D]
        vv = v[pages, :, at % page]
        qq = q[r].reshape(Hkv, -1, D)
        s = np.einsum("hgd,nhd->hgn", qq, kk) * scale
        mag = np.einsum("hgd,nhd->hgn", np.abs(qq), np.abs(kk)) * abs(scale)
        if softcap:
            s = softcap * np.tanh(s / softcap)
        m = s.max(-1, keepdims=True)
        p = np.exp(s - m)
        l = p.sum(-1, keepdims=True)
        p = p / l
        out[r] = np.einsum("hgn,nhd->hgd", p, vv).reshape(Hq, D)
        omag[r] = np.einsum("hgn,nhd->hgd", p, np.abs(vv)).reshape(Hq, D)
        lse[r] = (m + np.log(l)).reshape(Hq)
        smag[r] = mag.max(-1).reshape(Hq)
    return out, lse, smag, omag, count


def score_err(smag, dim, softcap=0.0):
    """fp32 product over dim and its scaling; the cap adds a few steps of a
    value of its own size (tanh to 2 ulp, two products)."""
    return (dim + 4) * U * smag + (8 * U * softcap if softcap else 0.0) + 4 * U * smag


def attention_tols(out, lse, smag, omag, count, dim, dtype, softcap=0.0):
    """Each weight is off by twice the largest score error (its own and the
    sum's), the exponential's 2^-22, the two-term split's 2^-16 and the sums'
    roundings (at most count additions, in 32 or more separate chains);
    the result is rounded to its type."""
    ds = score_err(smag, dim, softcap)[..., None]
    # exponents are formed in log2 units up to |score| * log2(e): one more rounding
    chain = (count[:, None, None] / 32 + 64) * U
    rel = 2 * (ds + 2.0 ** -22 + chain + 4 * U * np.abs(lse[..., None])) + 2.0 ** -16
    rel = np.where(np.isfinite(rel), rel, 0.0)
    err = rel * omag
    hs = HALF_STEP[dtype]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0  # half of fp16's smallest step
    tol_out = hs * (np.abs(out) + err) + err + tiny
    tol_lse = (ds + chain + 2.0 ** -22)[..., 0] + 4 * U * np.abs(lse)
    return tol_out, np.where(np.isfinite(tol_lse), tol_lse, 0.0)


def check_attention(got, got_lse, ref, dim, dtype, softcap=0.0, what=""):
    out, lse, smag, omag, count = ref
    tol, tol_lse = attention_tols(out, lse, smag, omag, count, dim, dtype, softcap)
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all(), f"{what}: {np.count_nonzero(~np.isfinite(g))} outputs not finite"
    bad = ~(np.abs(g - out) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outputs off; worst "
                           f"{np.max(np.abs(g - out) / np.maximum(tol, 1e-300)):.3g} tolerances, "
                           f"first at {tuple(int(x[0]) for x in np.nonzero(bad))}")
    if got_lse is not None:
        gl = got_lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(gl), np.isneginf(lse)), f"{what}: empty rows of lse"
        live = np.isfinite(lse)
        d = np.abs(gl[live] - lse[live])
        assert (d <= tol_lse[live]).all(), f"{what}: lse off by {(d / tol_lse[live]).max():.3g} tolerances"


# ------------------------------------------------------------------ inputs

def make_paged(gen, num_blocks, heads, page, dim, dtype, order="hnd", scale=1.0):
    """A cache [num_blocks, heads, page, dim] of N(0, scale) values in memory
    order hnd (heads of a page one after the other) or nhd (its tokens)."""
    x = torch.randn(num_blocks, heads, page, dim, generator=gen) * scale
    x = x.to(dtype)
    if order == "nhd":
        if dtype == torch.float8_e4m3fn:
            x = x.view(torch.uint8).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3).view(dtype)
        else:
            x = x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    return x


def to64(x):
    return x.float().double().numpy()


def make_block_table(rng, lens, page, num_blocks, max_blocks):
    """Distinct random pages per request; entries past a context are poison
    ids outside the cache (never to be read)."""
    B = len(lens)
    need = [-(-max(0, n) // page) for n in lens]
    perm = rng.permutation(num_blocks)
    assert sum(need) <= num_blocks
    bt = np.full((B, max_blocks), 2**31 - 1, np.int32)
    at = 0
    for b, n in enumerate(need):
        n = min(n, max_blocks)
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt


def poison_unseen(cache, bt, lens, page):
    """NaN in every cache row that no context covers (8-bit: the NaN code)."""
    seen = np.zeros((cache.shape[0], page), bool)
    for b, n in enumerate(lens):
        for p in range(max(0, n)):
            i = p // page
            if i < bt.shape[1] and 0 <= bt[b, i] < cache.shape[0]:
                seen[bt[b, i], p % page] = True
    blocks, offs = np.nonzero(~seen)
    if cache.dtype == torch.float8_e4m3fn:
        cache.view(torch.uint8)[blocks, :, offs] = 0x7F
    else:
        cache[blocks, :, offs] = float("nan")
