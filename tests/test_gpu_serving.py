"""GPU parity of the step plan, the rotary tables and the q/k norm + rotary +
cache insert with their plain 64-bit forms."""
import numpy as np
import pytest
import torch

import serving_testutil as su

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def idx():
    from sparse_attention_indexer_quant_gb300 import binding
    binding.check_device(torch.cuda.current_device())
    return binding


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ step plan

def run_plan(idx, cached, new, bt, free, head, num_tokens, num_blocks, page):
    errs = idx.new_errors()
    dbt = i32(bt)
    p = idx.plan_step(i32(cached), i32(new), dbt, i32(free), i32([head]), num_tokens, num_blocks,
                      page_size=page, errors=errs)
    torch.cuda.synchronize()
    want = su.ref_plan(cached, new, bt, np.asarray(free), head, num_tokens, num_blocks, page)
    for got, ref, name in zip(p[:5], want[:5], p._fields):
        assert np.array_equal(got.cpu().numpy(), ref), name
    assert p.pool_head.item() == want[5]
    assert np.array_equal(dbt.cpu().numpy(), want[6])
    assert errs.cpu().tolist() == [want[7], 0]


@pytest.mark.parametrize("B,page,new_hi,pad", [(1, 64, 1, 0), (1, 16, 700, 5), (7, 32, 40, 0),
                                               (255, 64, 1, 1), (256, 128, 1, 0),
                                               (1025, 16, 3, 100), (3000, 64, 2, 0),
                                               (40, 64, 3000, 777)])
def test_plan_step(idx, B, page, new_hi, pad):
    r = np.random.default_rng(B * 1000 + page)
    cached = r.integers(0, 2000, B)
    new = r.integers(0, new_hi + 1, B) if B > 1 else np.array([new_hi])
    have = -(-cached // page)
    need = -(-(cached + new) // page) - have
    num_blocks = int(have.sum() + need.sum()) + 10
    perm = r.permutation(num_blocks)
    max_blocks = int((have + need).max()) + 2
    bt = np.full((B, max_blocks), -9, np.int32)
    at = 0
    for b in range(B):
        bt[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    head = 3
    free = np.concatenate([[10**6] * head, perm[at:]]).astype(np.int32)
    run_plan(idx, cached, new, bt, free, head, int(new.sum()) + pad, num_blocks, page)


@pytest.mark.parametrize("case", ["no requests", "nothing new", "list runs out", "empty list",
                                  "bad pages", "negative", "past the table", "past the arrays",
                                  "head out of range", "overflow"])
def test_plan_step_edges(idx, case):
    page, num_blocks = 16, 64
    cached, new, head, num_tokens = [5, 16, 0, 40], [20, 1, 33, 0], 0, 54
    bt = np.full((4, 8), -1, np.int32)
    bt[0, 0], bt[1, 0], bt[3, :3] = 11, 12, [13, 14, 15]
    free = [20, 21, 22, 23, 24, 25, 26]
    if case == "no requests":
        cached, new, bt, num_tokens = [], [], np.zeros((0, 8), np.int32), 3
    if case == "nothing new":
        new, num_tokens = [0, 0, 0, 0], 0
    if case == "list runs out":
        free = free[:3]
    if case == "empty list":
        free = []
    if case == "bad pages":
        free[1], free[3], bt[0, 0] = -1, 64, 99
    if case == "negative":
        cached, new, num_tokens = [-1, 16, 0, 40], [20, -3, 33, 0], 40
    if case == "past the table":
        bt = bt[:, :3].copy()
        new, num_tokens = [90, 1, 33, 5], 129
    if case == "past the arrays":
        num_tokens = 30
    if case == "head out of range":
        head = 99
    if case == "overflow":
        cached, new, num_tokens = [5, 16, 0, 2**31 - 2], [20, 1, 33, 9], 54
    run_plan(idx, np.array(cached, np.int64), np.array(new, np.int64), bt, free, head, num_tokens,
             num_blocks, page)


def test_plan_step_writes_into_an_earlier_plan_and_a_graph_replays(idx):
    B, page, num_blocks = 5, 16, 200
    cached, new = i32([3, 16, 31, 0, 100]), i32([1] * B)
    bt = torch.zeros((B, 16), dtype=torch.int32, device="cuda")
    free, head = i32(np.arange(100, 200)), i32([0])
    plan = idx.plan_step(cached, new, bt, free, head, B, num_blocks, page_size=page)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx.plan_step(cached, new, bt, free, head, B, num_blocks, page_size=page, out=plan)
        cached.copy_(plan.context_lens)
        head.copy_(plan.pool_head)
    ref_bt, ref_cached, ref_head = bt.cpu().numpy(), cached.cpu().numpy(), 0
    for _ in range(40):
        g.replay()
        want = su.ref_plan(ref_cached, [1] * B, ref_bt, np.arange(100, 200), ref_head, B,
                           num_blocks, page)
        ref_cached, ref_head, ref_bt = want[0], want[5], want[6]
        torch.cuda.synchronize()
        assert np.array_equal(plan.slot_mapping.cpu().numpy(), want[2])
    assert head.item() == ref_head and np.array_equal(bt.cpu().numpy(), ref_bt)


def test_plan_step_refuses_one_word_for_both_heads(idx):
    head = i32([0])
    p = idx.plan_step(i32([1]), i32([1]), i32([[0]]), i32([1]), head, 1, 4)
    with pytest.raises(idx.IdxError):
        idx.plan_step(i32([1]), i32([1]), i32([[0]]), i32([1]), p.pool_head, 1, 4, out=p)


# ------------------------------------------------------------------ rotary tables

@pytest.mark.parametrize("kw", [dict(num_pos=1, rot=2), dict(num_pos=70, rot=64),
                                dict(num_pos=33, rot=6), dict(num_pos=1000, rot=256),
                                dict(num_pos=300, rot=10, pos0=12345),
                                dict(num_pos=2000, rot=128, pos0=1_000_000),
                                dict(num_pos=64, rot=64, pos0=2**31 - 64),
                                dict(num_pos=5000, rot=64, base=500000.0),
                                dict(num_pos=999, rot=64, scaling="linear", factor=4.0),
                                dict(num_pos=999, rot=128, scaling="ntk", factor=8.0),
                                dict(num_pos=70000, rot=64, scaling="yarn", factor=16.0,
                                     orig_len=4096, mscale=1.25),
                                dict(num_pos=100, rot=4, scaling="yarn", factor=2.0, orig_len=64),
                                dict(num_pos=100, rot=64, scaling="linear", factor=0.25)])
def test_rope_table(idx, kw):
    kw = dict(kw)
    n, rot, pos0, mscale = kw.pop("num_pos"), kw.pop("rot"), kw.pop("pos0", 0), kw.pop("mscale", None)
    cos, sin = idx.rope_table(n, rot, pos0=pos0, mscale=mscale, **kw)
    torch.cuda.synchronize()
    m = mscale or 1.0
    if kw.get("scaling") == "yarn" and mscale is None:
        m = 0.1 * np.log(kw["factor"]) + 1.0
    c, s = su.ref_table(pos0, n, rot, mscale=m, **kw)
    # the remainder of at most an eighth of a turn as fp32 (2^-24 relative), the
    # function's 2 ulp, mscale's and the product's rounding, 2^-33 turn of fixed
    # point, and the frequency's fp64 rounding (pow 1 ulp and three operations)
    tol = m * (np.pi / 4 * su.U + 5 * su.U + 2 * np.pi * 2.0 ** -33
               + (pos0 + n) * 5 * 2.0 ** -53 * max(1.0, 1 / kw.get("factor", 1.0)))
    assert np.abs(cos.cpu().numpy() - c).max() <= tol
    assert np.abs(sin.cpu().numpy() - s).max() <= tol


def test_rope_table_into_unaligned_and_empty_outputs(idx):
    ref = idx.rope_table(9, 8)
    buf = torch.full((2, 1 + 9 * 4 + 1), 7.0, device="cuda")
    cos, sin = buf[0, 1:37].view(9, 4), buf[1, 1:37].view(9, 4)
    idx.rope_table(9, 8, out=(cos, sin))
    torch.cuda.synchronize()
    assert torch.equal(cos, ref[0]) and torch.equal(sin, ref[1])
    assert (buf[:, 0] == 7).all() and (buf[:, 37] == 7).all()
    assert idx.rope_table(0, 8)[0].shape == (0, 4)


# ------------------------------------------------------------------ norm, turn, insert

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


def run_insert(idx, N, Hq, Hkv, D, rot, interleaved, dtype, cache, page, norm=True, pad=0,
               order="hnd", fused=True, scales=True, seed=0, in_place=False):
    g = torch.Generator().manual_seed(seed + N * 7 + D)
    dt, ct = TYPES[dtype], TYPES[cache]
    if fused:
        qkv = torch.randn(N, Hq + 2 * Hkv, D, generator=g).to(dt).cuda()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:  # head-major tensors seen token by token
        q, k, v = (torch.randn(h, N, D, generator=g).to(dt).cuda().transpose(0, 1)
                   for h in (Hq, Hkv, Hkv))
    if in_place:
        q = q.contiguous()
    num_blocks = -(-N // page) + 3
    slots = torch.randperm(num_blocks * page, generator=g)[:N]
    slots[torch.randperm(N, generator=g)[:pad]] = -1
    num_pos = 300
    pos = torch.randint(0, num_pos, (N,), generator=g, dtype=torch.int32)
    ang = torch.rand(num_pos, rot // 2, generator=g, dtype=torch.float64) * 6.3
    cos, sin = ang.cos().float(), ang.sin().float()
    qw = kw = None
    if norm:
        qw, kw = (1 + 0.3 * torch.randn(D, generator=g) for _ in range(2))
    ks = vs = None
    if cache == "e4m3" and scales:
        ks, vs = (0.01 + 0.05 * torch.rand(Hkv, generator=g) for _ in range(2))
    kc, vc = (su.make_paged(g, num_blocks, Hkv, page, D, ct, order) for _ in range(2))
    before = su.to64(kc), su.to64(vc)
    kc, vc = kc.cuda(), vc.cuda()
    if order == "nhd":
        assert kc.stride(2) == Hkv * D
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    q64, k64, v64 = (su.to64(x.cpu()) for x in (q, k, v))
    errs = idx.new_errors()
    out = idx.qk_norm_rope_insert(q, k, v, c(qw), c(kw), 1e-6, pos.cuda(), cos.cuda(), sin.cuda(),
                                  rot, slots.cuda(), kc, vc, interleaved=interleaved,
                                  k_scale=c(ks), v_scale=c(vs), errors=errs,
                                  q_out=q if in_place else None)
    torch.cuda.synchronize()
    assert errs.cpu().tolist() == [0, 0]
    cs, sn = cos.double().numpy()[pos.numpy()], sin.double().numpy()[pos.numpy()]
    eps = float(np.float32(1e-6))

    def close(got, ref, mag, normed, what):
        tol = su.turned_tol(ref, mag, D, normed, su.HALF_STEP[dt], 2.0 ** -25 if dtype == "fp16" else 0)
        assert (np.abs(got - ref) <= tol).all(), f"{what}: {(np.abs(got - ref) / tol).max()}"

    ref, mag = su.ref_turned(q64, None if qw is None else qw.double().numpy(), eps, cs, sn, rot,
                             interleaved)
    close(su.to64(out.cpu()), ref, mag, norm, "q")
    kref, kmag = su.ref_turned(k64, None if kw is None else kw.double().numpy(), eps, cs, sn, rot,
                               interleaved)
    keep = slots.numpy() >= 0
    at = slots.numpy()[keep]
    for got, ref, mag, old, scale, what in (
            (su.to64(kc.cpu()), kref, kmag, before[0], ks, "k"),
            (su.to64(vc.cpu()), v64, np.abs(v64), before[1], vs, "v")):
        rows = got[at // page, :, at % page]
        ref, mag = ref[keep], mag[keep]
        if cache == "e4m3":
            s = scale.double().numpy()[:, None] if scale is not None else 1.0
            want = np.clip(ref / s, -su.E4M3_MAX, su.E4M3_MAX)
            err = (D + 14) * su.U * mag / s if what == "k" else 2 * su.U * mag / s
            # half a step of a normal value (2^-4 relative) or of a subnormal (2^-10)
            tol = np.maximum(2.0 ** -4 * (np.abs(want) + err), 2.0 ** -10) + err
            assert (np.abs(rows - want) <= tol).all(), what
            if what == "v":  # no arithmetic but the division: the very codes of the nearest values
                exact = torch.from_numpy((v64[keep].astype(np.float32)
                                          / (s if scale is None else s.astype(np.float32))))
                exact = exact.clamp(-su.E4M3_MAX, su.E4M3_MAX).to(torch.float8_e4m3fn)
                assert np.array_equal(rows, su.to64(exact))
        elif what == "v":
            assert np.array_equal(rows, ref)
        else:
            close(rows, ref, mag, norm, what)
        untouched = np.ones((num_blocks, page), bool)
        untouched[at // page, at % page] = False
        b, o = np.nonzero(untouched)
        assert np.array_equal(got[b, :, o], old[b, :, o]), f"{what}: rows outside the slots changed"


@pytest.mark.parametrize("N,Hq,Hkv,D,rot,inter,dtype,cache,page,kw", [
    (1, 1, 1, 64, 64, False, "bf16", "bf16", 16, {}),
    (1, 32, 8, 128, 128, True, "bf16", "bf16", 64, {}),
    (33, 24, 4, 128, 64, False, "fp16", "fp16", 64, {}),
    (77, 5, 5, 256, 96, False, "bf16", "e4m3", 32, dict(pad=3)),
    (50, 6, 2, 64, 30, True, "fp16", "e4m3", 128, dict(order="nhd")),
    (50, 6, 3, 256, 2, True, "bf16", "bf16", 16, dict(norm=False)),
    (40, 4, 1, 128, 0, False, "bf16", "bf16", 16, {}),
    (40, 4, 1, 128, 0, True, "fp16", "e4m3", 16, dict(scales=False)),
    (700, 16, 4, 64, 48, False, "bf16", "bf16", 64, dict(fused=False, order="nhd")),
    (3000, 32, 8, 128, 128, False, "bf16", "bf16", 64, dict(pad=17)),
    (3001, 31, 7, 64, 62, True, "fp16", "fp16", 64, dict(fused=False)),
    (2500, 9, 3, 256, 256, False, "fp16", "e4m3", 64, {}),
    (130, 8, 2, 128, 64, False, "bf16", "bf16", 64, dict(in_place=True)),
])
def test_qk_norm_rope_insert(idx, N, Hq, Hkv, D, rot, inter, dtype, cache, page, kw):
    run_insert(idx, N, Hq, Hkv, D, rot, inter, dtype, cache, page, **kw)


def test_insert_skips_and_counts(idx):
    N, Hq, Hkv, D, page, nb = 8, 2, 1, 64, 16, 2
    q, k, v = (torch.ones(N, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    cos, sin = torch.ones(4, 8, device="cuda"), torch.zeros(4, 8, device="cuda")
    pos = i32([0, 1, 2, 3, -1, 4, 2, 2])           # 4 and 5 are off the table
    slots = torch.tensor([0, 1, -1, 32, 4, 5, -2, 31], device="cuda")  # 3 and 6 off the cache
    kc, vc = idx.new_kv_cache(nb, Hkv, D, page_size=page)
    out = torch.full((N, Hq, D), -5.0, dtype=torch.bfloat16, device="cuda")
    errs = idx.new_errors()
    idx.qk_norm_rope_insert(q, k, v, None, None, 0.0, pos, cos, sin, 16, slots, kc, vc, q_out=out,
                            errors=errs)
    torch.cuda.synchronize()
    assert errs.cpu().tolist() == [4, 0]
    written = (out == 1).all(-1).all(-1).cpu().tolist()
    assert written == [True, True, True, True, False, False, True, True]
    assert (out[4:6] == -5).all()
    filled = (kc[:, 0, :, 0] == 1).reshape(-1).nonzero().flatten().cpu().tolist()
    assert filled == [0, 1, 31] and torch.equal(kc, vc)


def test_insert_keeps_infinities_in_their_dimension(idx):
    """A dimension that does not turn is not multiplied by anything."""
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 40], q[0, 0, 41] = float("inf"), float("-inf")
    kc, vc = idx.new_kv_cache(1, 1, 64, page_size=16)
    t = torch.full((1, 16), 0.5, device="cuda")
    for inter in (False, True):
        out = idx.qk_norm_rope_insert(q, q, q, None, None, 0.0, i32([0]), t, t, 32,
                                      torch.zeros(1, dtype=torch.int64, device="cuda"), kc, vc,
                                      interleaved=inter)
        torch.cuda.synchronize()
        assert torch.equal(out, q) and torch.equal(kc[0, 0, 0], q[0, 0]) and torch.equal(vc, kc)


@pytest.mark.parametrize("inter", [False, True])
def test_insert_takes_tables_and_weights_at_any_address(idx, inter):
    """4-byte aligned tables and weights give the same bytes as aligned ones."""
    q = torch.randn(37, 3, 128, device="cuda").bfloat16()
    cos, sin, w = torch.rand(50, 32, device="cuda"), torch.rand(50, 32, device="cuda"), torch.rand(128, device="cuda")

    def off(t):
        buf = torch.empty(t.numel() + 1, device="cuda")
        buf[1:].copy_(t.flatten())
        return buf[1:].view(t.shape)

    pos, slots = i32(np.arange(37) % 50), torch.arange(37, device="cuda")
    got = []
    for f in (lambda t: t, off):
        kc, vc = idx.new_kv_cache(3, 3, 128, page_size=16)
        out = idx.qk_norm_rope_insert(q, q, q, f(w), f(w), 1e-6, pos, f(cos), f(sin), 64, slots, kc,
                                      vc, interleaved=inter)
        got.append((out, kc, vc))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_insert_on_another_stream(idx):
    s = torch.cuda.Stream()
    q = torch.randn(64, 8, 128, device="cuda").bfloat16()
    kc, vc = idx.new_kv_cache(2, 8, 128)
    slots = torch.arange(64, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    out = idx.qk_norm_rope_insert(q, q, q, None, None, 0.0, None, None, None, 0, slots, kc, vc,
                                  stream=s)
    s.synchronize()
    assert torch.equal(out, q) and torch.equal(vc[0].transpose(0, 1), q)


def test_insert_no_tokens(idx):
    kc, vc = idx.new_kv_cache(2, 1, 64)
    e = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    out = idx.qk_norm_rope_insert(e, e, e, None, None, 0.0, i32([]), None, None, 0,
                                  torch.empty(0, dtype=torch.int64, device="cuda"), kc, vc)
    assert out.shape == (0, 1, 64)
