"""Shapes by the way in which the paged attention shares them out, and problems of
many distinct kv heads in little memory.

A call takes its items whole, by teams of 8, 4, 2 or 1 warps, or splits them
(idx_paged_attention_form).  A split call cuts the batch's units into segments,
which depends on the lengths too: `cut` follows csrc/paged_attn.cuh's Cut."""
import collections

import numpy as np
import torch

import serving_testutil as su

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
SETUP, MIN_SEGMENT, LEVELS = 3, 5, 5

Split = collections.namedtuple("Split", "way segments levels")


def cut(form, lens, next_n, heads, topk=0, window=0):
    """How a split call of these lengths is cut: pieces of items, equal segments
    over the batch, or levels of segments that the CTAs claim."""
    HR, R = heads * form.row_tiles, form.places
    units = []
    for n in lens:
        first = max(0, n - next_n + 1 - window) if window else 0
        units.append(max(1, -(-n // form.unit) - first // form.unit))
    if topk:
        units = [-(-topk // form.unit)] * (len(lens) * next_n)
    U = sum(u + SETUP for u in units) * HR
    K = max([k for k in range(2, LEVELS) if U >> (k + 1) >= MIN_SEGMENT * R], default=0)
    if K:
        return Split("claimed", R * (K + 1), K + 1)
    real = sum(units) * HR
    q0 = -(-real // R)
    step = max(1, q0 // 12)
    for j in range(4):
        pieces = sum(-(-u // (q0 + j * step)) for u in units)
        if pieces <= R // HR:
            return Split("pieces", pieces * HR, 1)
    return Split("equal", min(R, U), 1)


class Problem:
    """kv head h's values lie h * step values after the first head's in every
    token's row: distinct heads in a cache little larger than one head's."""

    def __init__(self, lens, heads, group, D, cache="bf16", next_n=1, page=64, topk=0, room=0,
                 listed=0.9, seed=0):
        dtype = "fp16" if cache == "fp16" else "bf16"
        g = torch.Generator().manual_seed(seed + 31 * len(lens) + D)
        r = np.random.default_rng(seed + 7)
        self.lens, self.heads, self.D, self.next_n = list(lens), heads, D, next_n
        self.dtype = TYPES[dtype]
        step = 16 if cache == "e4m3" else 8
        need = sum(-(-n // page) for n in lens)
        blocks, mb = need + 2, max(1, -(-max(max(lens), room) // page))
        self.bt = su.make_block_table(r, lens, page, blocks, mb)
        width = -(-(D + step * (heads - 1)) // 16) * 16
        rows = len(lens) * next_n
        self.q = (torch.randn(rows, heads * group, D, generator=g) * 2).to(self.dtype)
        ct = TYPES[cache]
        self.base = [torch.randn(blocks, 1, page, width, generator=g).to(ct) for _ in range(2)]
        self.base64 = [x.float().double()[:, 0] for x in self.base]
        self.step, self.page = step, page
        self.scales = None
        if cache == "e4m3":
            self.scales = [0.3 + torch.rand(heads, generator=g) for _ in range(2)]
        self.topk = None
        if topk:
            self.topk = np.full((rows, topk), -1, np.int64)
            for i in range(rows):
                end = max(0, lens[i // next_n] - next_n + 1 + i % next_n)
                m = min(int(topk * listed), end)
                self.topk[i, r.permutation(topk)[:m]] = r.permutation(end)[:m]
        for x in self.base:
            su.poison_unseen(x, self.bt, lens, page)
        self.form_args = (len(lens), next_n, heads * group, heads, D, ct, page, mb, topk)

    def caches(self):
        out = []
        for x in self.base:
            d = x.cuda()
            s = d.stride()
            out.append(d.as_strided((d.shape[0], self.heads, self.page, self.D),
                                    (s[0], self.step, s[2], 1)))
        return out

    def on_gpu(self):
        """Arguments of paged_attention, without scale, cap and window."""
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
        k, v = self.caches()
        kw = dict(topk=None if self.topk is None else i32(self.topk), return_lse=True)
        if self.scales:
            kw["k_scale"], kw["v_scale"] = (x.cuda() for x in self.scales)
        return (self.q.cuda(), k, v, i32(self.bt), i32(self.lens), self.next_n), kw

    def reference(self, softcap=0.0, window=0, lens=None):
        """As serving_testutil.ref_attention, head by head in 64 bits."""
        lens = self.lens if lens is None else lens
        R, Hq, D = self.q.shape
        H, f32 = self.heads, np.float32
        scale = float(f32(D ** -0.5))
        out, omag = (np.zeros((R, Hq, D)) for _ in range(2))
        lse, smag = np.full((R, Hq), -np.inf), np.zeros((R, Hq))
        count = np.zeros(R, np.int64)
        ks = vs = [1.0] * H
        if self.scales:
            ks, vs = (x.double() for x in self.scales)
        for row in range(R):
            b, end = row // self.next_n, max(0, lens[row // self.next_n] - self.next_n + 1 + row % self.next_n)
            if self.topk is not None:
                at = self.topk[row][(self.topk[row] >= 0) & (self.topk[row] < end)]
            else:
                at = np.arange(max(0, end - window) if window else 0, end)
            count[row] = len(at)
            if not len(at):
                continue
            pages, offs = torch.from_numpy(self.bt[b][at // self.page].astype(np.int64)), torch.from_numpy(at % self.page)
            rows = [x[pages, offs] for x in self.base64]  # [n, width]
            G = Hq // H
            for h in range(H):
                k, v = (x[:, h * self.step:h * self.step + D] for x in rows)
                k, v = k * ks[h], v * vs[h]
                q = self.q[row, h * G:(h + 1) * G].double()
                s = q @ k.T * scale
                mag = q.abs() @ k.abs().T * scale
                if softcap:
                    s = softcap * torch.tanh(s / softcap)
                m = s.amax(-1, keepdim=True)
                p = torch.exp(s - m)
                total = p.sum(-1, keepdim=True)
                p = p / total
                at = slice(h * G, (h + 1) * G)
                out[row, at], omag[row, at] = (p @ v).numpy(), (p @ v.abs()).numpy()
                lse[row, at] = (m + torch.log(total))[:, 0].numpy()
                smag[row, at] = mag.amax(-1).numpy()
        return out, lse, smag, omag, count


def ragged(seed, n, most, first=(0,)):
    r = np.random.default_rng(seed)
    return list(first) + r.integers(0, most + 1, n - len(first)).tolist()


# Split calls by the way they are cut on 152 SMs (Problem's arguments): claimed segments
# over hundreds of requests with empty ones among them, over a few long ones, with
# selections; equal segments that cross items; pieces of items.
WAYS = {
    "claimed, 320 requests": ("claimed", dict(lens=ragged(0, 320, 300, (0, 0, 300, 1)), heads=16, group=2,
                                              D=64, room=40000)),
    "claimed, 320 requests, E4M3, 2 tokens": ("claimed", dict(lens=ragged(1, 320, 300, (0, 1, 2, 300)), heads=16,
                                                              group=1, D=128, cache="e4m3", next_n=2, page=16,
                                                              room=40000)),
    "claimed, 300 requests, fp16, 12 rows": ("claimed", dict(lens=ragged(2, 300, 200, (0, 200)), heads=16, group=6,
                                                             D=128, cache="fp16", next_n=2, page=16, room=40000)),
    "claimed, few long": ("claimed", dict(lens=[9000, 0, 4000, 1, 2500, 130], heads=64, group=1, D=256)),
    "claimed, selections": ("claimed", dict(lens=[5000, 100, 0] + [2500] * 37, heads=8, group=2, D=256,
                                            cache="e4m3", next_n=2, topk=2048)),
    "equal, ragged": ("equal", dict(lens=[3000, 1, 0], heads=160, group=4, D=128, room=9000)),
    "equal, few long": ("equal", dict(lens=[9000, 0, 4000, 1, 2500, 130], heads=64, group=1, D=64)),
    "equal, selections": ("equal", dict(lens=[5000, 4500, 100, 0, 4100, 4999, 4001, 4000], heads=13, group=1,
                                        D=128, topk=4000)),
    "equal, selections, 20 rows": ("equal", dict(lens=[5000], heads=80, group=20, D=128, topk=3000)),
    "pieces, ragged": ("pieces", dict(lens=[9000, 100, 7000, 0], heads=4, group=3, D=64, next_n=2)),
    "pieces, selections": ("pieces", dict(lens=[9000], heads=4, group=1, D=64, topk=4000)),
}


def way_of(idx, problem, lens=None, sms=None):
    form = idx.paged_attention_form(*problem.form_args, sms=sms)
    lens = problem.lens if lens is None else lens
    return cut(form, lens, problem.next_n, problem.heads, problem.form_args[-1]).way if form.split else "whole"


# Shapes of whole and split calls for every kernel: (requests, kv heads, keys) tried in
# this order until one is shared out as asked for.
GROUPS = {"several": {1: (3, 2), 2: (6, 2), 4: (10, 2)},  # row tiles: heads a kv head, tokens
          "one": {1: (5, 1), 2: (13, 1), 4: (24, 1)}, "listed": {1: (5, 1), 2: (13, 1), 4: (24, 1)}}
SHAPES = [(2, 1, 4000), (2, 1, 2000), (2, 2, 700), (3, 2, 300), (2, 1, 200), (20, 10, 300), (20, 16, 96),
          (5, 40, 300), (2, 160, 96), (40, 8, 300), (80, 8, 96), (80, 8, 48), (40, 20, 96), (160, 8, 96),
          (160, 8, 48), (160, 8, 16), (320, 8, 40), (320, 8, 16), (320, 10, 16)]


def shape_for(idx, D, cache, tiles, sights, warps, sms=None):
    """Problem's arguments of a call that is shared out by `warps` (0: split); sights:
    one new token a request, several, or selections."""
    group, next_n = GROUPS[sights][tiles]
    listed = sights == "listed"
    for B, heads, keys in SHAPES:
        if heads * group > 4096:
            continue
        room = 20000 if warps == 0 and not listed else keys
        f = idx.paged_attention_form(B, next_n, heads * group, heads, D, TYPES[cache], 16, -(-room // 16),
                                     keys if listed else 0, sms=sms)
        if (0 if f.split else f.warps) == warps:
            lens = ragged(D + tiles, B, 2 * keys if listed else keys, (keys, 0)[:min(B, 2)])
            return dict(lens=lens, heads=heads, group=group, D=D, cache=cache, next_n=next_n, page=16,
                        topk=keys if listed else 0, room=room)
    return None


FORMS = [(D, cache, tiles, sights, warps) for D in (64, 128, 256) for cache in TYPES
         for tiles in ((1, 2, 4) if D < 256 else (1, 2)) for sights in GROUPS
         for warps in (0, 8, 4, 2, 1)]
