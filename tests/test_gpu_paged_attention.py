"""GPU parity of the paged attention with its plain 64-bit form: types, head
layouts, lengths around every tile and page edge, windows, caps, selections,
split and joined items, poisoned memory, bad pages, streams and graphs."""
import numpy as np
import pytest
import torch

import serving_testutil as su

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def idx():
    from sparse_attention_indexer_quant_gb300 import binding
    binding.check_device(torch.cuda.current_device())
    return binding


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def make(lens, Hq, Hkv, D, dtype="bf16", cache="bf16", page=64, next_n=1, order="hnd", k=0,
         extra_blocks=0, seed=0, q_order="tokens", scales=True, hole=0.2, peak=2.0):
    """One problem on the CPU: dict of tensors and the 64-bit reference's inputs."""
    g = torch.Generator().manual_seed(seed + 31 * len(lens) + D)
    r = np.random.default_rng(seed + 7)
    need = sum(-(-max(0, n) // page) for n in lens)
    blocks = need + 2
    mb = max(1, max(-(-max(0, n) // page) for n in lens)) + extra_blocks
    bt = su.make_block_table(r, lens, page, blocks, mb)
    R = len(lens) * next_n
    q = (torch.randn(R, Hq, D, generator=g) * peak).to(TYPES[dtype])
    if q_order == "heads":
        q = q.transpose(0, 1).contiguous().transpose(0, 1)
    kc, vc = (su.make_paged(g, blocks, Hkv, page, D, TYPES[cache], order) for _ in range(2))
    ks = vs = None
    k64, v64 = su.to64(kc), su.to64(vc)
    if cache == "e4m3" and scales:
        ks, vs = (0.3 + torch.rand(Hkv, generator=g) for _ in range(2))
        k64 = k64 * ks.double().numpy()[None, :, None, None]
        v64 = v64 * vs.double().numpy()[None, :, None, None]
    topk = None
    if k:
        topk = np.full((R, k), -1, np.int64)
        for row in range(R):
            end = max(0, lens[row // next_n] - next_n + 1 + row % next_n)
            m = min(k, end)
            topk[row, :m] = r.permutation(end)[:m]
            holes = r.random(k) < hole
            topk[row, holes] = -1
    su.poison_unseen(kc, bt, lens, page)
    su.poison_unseen(vc, bt, lens, page)
    return dict(q=q, kc=kc, vc=vc, bt=bt, lens=lens, next_n=next_n, ks=ks, vs=vs, topk=topk,
                k64=k64, v64=v64, D=D, dtype=TYPES[dtype])


def call(idx, p, scale=None, softcap=0.0, window=0, errs=None, **kw):
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    q = p["q"]
    dq = q.cuda()
    assert dq.stride() == q.stride()
    dk, dv = p["kc"].cuda(), p["vc"].cuda()
    assert dk.stride() == p["kc"].stride()
    return idx.paged_attention(dq, dk, dv, i32(p["bt"]), i32(p["lens"]), p["next_n"], scale=scale,
                               softcap=softcap, window=window,
                               topk=None if p["topk"] is None else i32(p["topk"]),
                               k_scale=c(p["ks"]), v_scale=c(p["vs"]), return_lse=True,
                               errors=errs, **kw)


def check(idx, p, scale=None, softcap=0.0, window=0, bad=0, what="", **kw):
    errs = idx.new_errors()
    out, lse = call(idx, p, scale, softcap, window, errs, **kw)
    torch.cuda.synchronize()
    assert errs.cpu().tolist() == [bad, 0]
    f32 = np.float32
    s = float(f32(p["D"] ** -0.5 if scale is None else scale))
    ref = su.ref_attention(su.to64(p["q"]), p["k64"], p["v64"], p["bt"], p["lens"], p["next_n"],
                           s, float(f32(softcap)), window, p["topk"])
    su.check_attention(out, lse, ref, p["D"], p["dtype"], softcap, what)
    return out, lse


EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"),
                                         ("fp16", "e4m3")])
def test_lengths_around_every_edge(idx, D, dtype, cache):
    check(idx, make(EDGES, 4, 2, D, dtype, cache, page=16))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("order", ["hnd", "nhd"])
def test_page_sizes_and_orders(idx, page, order):
    check(idx, make([1, 129, 700, 1111, 2049], 8, 4, 128, page=page, order=order, q_order="heads"))
    check(idx, make([1, 129, 700, 1111], 6, 2, 64, "fp16", "e4m3", page=page, order=order))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (5, 1), (8, 8), (12, 4), (16, 1), (17, 1),
                                    (32, 1), (33, 1), (64, 1), (40, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_head_groups(idx, Hq, Hkv, D):
    check(idx, make([5, 1000, 130], Hq, Hkv, D, page=32))


@pytest.mark.parametrize("next_n", [2, 3, 5, 16])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_several_new_tokens(idx, next_n, cache):
    lens = [0, 1, 2, next_n - 1, next_n, next_n + 1, 16, 17, 128, 129, 1000, 3001]
    check(idx, make(lens, 8, 2, 128, "bf16", cache, page=16, next_n=next_n))
    check(idx, make(lens, 8, 2, 64, "bf16", cache, page=16, next_n=next_n), window=100)


@pytest.mark.parametrize("window", [1, 2, 16, 100, 127, 128, 129, 1000, 5000, 2**31 - 1])
def test_windows(idx, window):
    check(idx, make(EDGES + [999, 1000, 1001, 4000], 4, 2, 128, page=16), window=window)
    check(idx, make([0, 1, 500, 4000, 2222], 6, 1, 256, "fp16", "fp16", next_n=3), window=window)


@pytest.mark.parametrize("cache", ["fp16", "e4m3"])
def test_cap_and_scale(idx, cache):
    p = make([1, 77, 300, 2500], 8, 2, 64, "fp16", cache, page=32, peak=6.0)
    check(idx, p, softcap=15.0, scale=0.3)
    check(idx, p, softcap=50.0, window=200)
    check(idx, p, scale=0.0)
    check(idx, p, scale=-0.25)


@pytest.mark.parametrize("k", [1, 7, 16, 128, 129, 500, 2048])
@pytest.mark.parametrize("D,dtype,cache,order", [(128, "bf16", "bf16", "nhd"),
                                                 (64, "fp16", "e4m3", "hnd"),
                                                 (256, "bf16", "e4m3", "nhd"),
                                                 (64, "bf16", "bf16", "hnd"),
                                                 (256, "fp16", "fp16", "hnd")])
def test_selections(idx, k, D, dtype, cache, order):
    check(idx, make([0, 1, 3, 130, 2500, 3000], 8, 2, D, dtype, cache, page=16, order=order, k=k))
    check(idx, make([1, 2, 700], 40, 2, D, dtype, cache, page=64, next_n=2, order=order, k=k,
                    hole=0.0), softcap=25.0)


def test_selection_repeats_and_positions_out_of_sight(idx):
    p = make([100, 40], 4, 2, 128, page=16, next_n=2, k=8, hole=0.0)
    p["topk"][0] = [98, 99, 100, 5, 5, 5, -1, 2**31 - 1]  # row 0 sees [0, 99)
    p["topk"][3] = [-5, -1, 39, 40, 0, 0, 1, 1]           # row 3 sees [0, 40)
    check(idx, p, bad=4)
    p["topk"][2] = -1                                     # nothing selected
    out, lse = check(idx, p, bad=4)
    assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()


@pytest.mark.parametrize("order", ["hnd", "nhd"])
def test_long_requests_are_split_and_joined(idx, order):
    check(idx, make([30000, 1, 77], 4, 1, 128, order=order))
    check(idx, make([9000], 16, 2, 64, "bf16", "e4m3", order=order, next_n=2))
    check(idx, make([20000], 8, 1, 256, "fp16", "fp16", page=128, order=order))


def test_many_requests(idx):
    r = np.random.default_rng(3)
    lens = r.integers(0, 400, 300).tolist()
    check(idx, make(lens, 4, 2, 64, page=16))
    check(idx, make(lens, 4, 2, 64, page=16, extra_blocks=100))  # same lengths, split launch
    check(idx, make(lens[:150], 4, 4, 128, "bf16", "e4m3", page=16, k=64, next_n=2))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"),
                                         ("fp16", "e4m3")])
@pytest.mark.parametrize("group", [1, 5, 12, 20, 40])
def test_many_short_requests(idx, D, dtype, cache, group):
    """Enough short items that each is a single warp's."""
    r = np.random.default_rng(D + group)
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 255, 256] + r.integers(0, 257, 310).tolist()
    check(idx, make(lens, 2 * group, 2, D, dtype, cache, page=16, seed=group))


@pytest.mark.parametrize("D,cache,order", [(64, "bf16", "nhd"), (128, "e4m3", "hnd"),
                                           (128, "bf16", "nhd"), (256, "bf16", "hnd")])
def test_many_short_rows_in_every_form(idx, D, cache, order):
    r = np.random.default_rng(D)
    lens = [0, 1, 2, 3, 100] + r.integers(0, 200, 215).tolist()
    check(idx, make(lens, 9, 3, D, "bf16", cache, page=32, next_n=3, order=order), softcap=20.0)
    check(idx, make(lens, 9, 3, D, "bf16", cache, page=32, next_n=3, order=order), window=37,
          scale=-0.1)
    check(idx, make(lens, 9, 3, D, "bf16", cache, page=64, next_n=2, k=100, order=order))
    check(idx, make(lens, 9, 3, D, "bf16", cache, page=16, next_n=1, k=256, order=order, hole=0.0))
    check(idx, make(lens, 9, 3, D, "bf16", cache, page=128, next_n=2, k=1, order=order))
    p = make(lens, 9, 3, D, "bf16", cache, page=16, order=order)
    p["bt"][4, 2], p["bt"][4, 3] = -7, 10**7   # 100 tokens: pages 0 - 6
    check(idx, p, bad=2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"),
                                         ("fp16", "e4m3")])
@pytest.mark.parametrize("heads,group", [(20, 4), (20, 12), (20, 24), (35, 4), (35, 20), (70, 3),
                                         (70, 11), (140, 1)])
def test_items_of_few_warps(idx, D, dtype, cache, heads, group):
    """400 to 2800 items of at most 96 keys, which teams of four, two or one
    warps take."""
    r = np.random.default_rng(heads + group)
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 95, 96] + r.integers(0, 97, 7).tolist()
    check(idx, make(lens, heads * group, heads, D, dtype, cache, page=32, seed=group))
    check(idx, make(lens, heads * group, heads, D, dtype, cache, page=16, k=96, hole=0.1), softcap=9.0)


@pytest.mark.parametrize("D,cache,next_n", [(64, "bf16", 1), (128, "bf16", 3), (128, "e4m3", 2),
                                            (256, "bf16", 1)])
def test_items_of_few_warps_in_every_form(idx, D, cache, next_n):
    """Lists of several tables of a team, windows, orders, bad pages."""
    r = np.random.default_rng(D)
    lens = [0, 1, 700, 701, 1000] + r.integers(300, 1000, 15).tolist()
    for heads, order in ((20 // next_n, "nhd"), (35, "hnd")):
        check(idx, make(lens, 3 * heads, heads, D, "bf16", cache, page=64, next_n=next_n, k=700,
                        order=order, hole=0.3))
        check(idx, make(lens, 3 * heads, heads, D, "bf16", cache, page=16, next_n=next_n,
                        order=order), window=77, scale=-0.1)
        p = make(lens, 3 * heads, heads, D, "bf16", cache, page=64, next_n=next_n, order=order)
        p["bt"][2, 2], p["bt"][2, 10] = -7, 10**7
        check(idx, p, softcap=20.0, bad=2)


def test_ranges_longer_than_the_page_table_in_shared_memory(idx):
    """A CTA's range of more than 32768 keys, and of more than 2048 listed
    positions: 320 kv heads that are one head seen again (head stride 0)."""
    p = make([50000], 320, 1, 64, page=128, seed=5)
    one = su.ref_attention(su.to64(p["q"]), p["k64"], p["v64"], p["bt"], p["lens"], 1, 0.125)
    kc, vc = (p[x].cuda().expand(-1, 320, -1, -1) for x in ("kc", "vc"))
    out, lse = idx.paged_attention(p["q"].cuda(), kc, vc, i32(p["bt"]), i32(p["lens"]), 1,
                                   return_lse=True)
    torch.cuda.synchronize()
    su.check_attention(out, lse, one, 64, torch.bfloat16)
    r = np.random.default_rng(4)
    topk = r.integers(0, 50000, (1, 9000))
    topk[0, r.random(9000) < 0.3] = -1
    one = su.ref_attention(su.to64(p["q"]), p["k64"], p["v64"], p["bt"], p["lens"], 1, 0.125,
                           topk=topk)
    out, lse = idx.paged_attention(p["q"].cuda(), kc, vc, i32(p["bt"]), i32(p["lens"]), 1,
                                   topk=i32(topk), return_lse=True)
    torch.cuda.synchronize()
    su.check_attention(out, lse, one, 64, torch.bfloat16)


def test_offsets_past_32_bits(idx):
    """Pages whose byte and element offsets pass 2^32."""
    D, Hkv, page, L = 128, 8, 64, 700
    nb = 70000
    kc, vc = (torch.empty(nb, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kc.numel() > 2**32
    p = make([L], 8, Hkv, D, page=page)
    far = np.arange(nb - p["kc"].shape[0], nb)
    kc[far[0]:], vc[far[0]:] = p["kc"].cuda(), p["vc"].cuda()
    bt = np.where(p["bt"] < p["kc"].shape[0], p["bt"] + far[0], p["bt"])
    ref = su.ref_attention(su.to64(p["q"]), p["k64"], p["v64"], p["bt"], [L], 1, float(np.float32(D ** -0.5)))
    out, lse = idx.paged_attention(p["q"].cuda(), kc, vc, i32(bt), i32([L]), 1, return_lse=True)
    topk = np.random.default_rng(0).permutation(L)[None, :300]
    out2, lse2 = idx.paged_attention(p["q"].cuda(), kc, vc, i32(bt), i32([L]), 1, topk=i32(topk),
                                     return_lse=True)
    torch.cuda.synchronize()
    su.check_attention(out, lse, ref, D, torch.bfloat16)
    ref = su.ref_attention(su.to64(p["q"]), p["k64"], p["v64"], p["bt"], [L], 1,
                           float(np.float32(D ** -0.5)), topk=topk)
    su.check_attention(out2, lse2, ref, D, torch.bfloat16)


def test_bad_pages_and_lengths_are_skipped_and_counted(idx):
    p = make([200, 64, 300], 4, 2, 128, page=16)
    p["bt"][0, 3], p["bt"][0, 12], p["bt"][2, 0] = -1, 10**6, 2**31 - 1
    check(idx, p, bad=3)
    check(idx, p, window=150, bad=2)   # request 0 sees [50, 200): pages 3 and 12; request 2 not page 0
    p = make([200, 64, 300], 4, 2, 128, page=16)
    p["lens"] = [200, -4, 10**6]       # none; more than the table's 19 pages
    p["kc"][int(p["bt"][2, 18])] = 0.5  # the last page is seen whole now
    p["vc"][int(p["bt"][2, 18])] = 0.25
    p["k64"][int(p["bt"][2, 18])], p["v64"][int(p["bt"][2, 18])] = 0.5, 0.25
    check(idx, p, bad=2)


def test_infinite_and_nan_values_stay_in_their_rows(idx):
    """Request 0's cache holds a NaN in sight; request 1 shares no page."""
    p = make([100, 100], 4, 2, 128, page=16)
    clean, _ = call(idx, p)
    p["vc"][int(p["bt"][0, 2]), 1, 3, 7] = float("nan")
    p["kc"][int(p["bt"][0, 1]), 0, 0] = float("inf")
    out, lse = call(idx, p)
    torch.cuda.synchronize()
    assert torch.equal(out[1], clean[1])
    assert torch.isnan(out[0, 2:, 7]).all() and torch.isfinite(out[0, 2:, :7]).all()
    assert not torch.isfinite(out[0, :2]).any()


def test_large_scores(idx):
    """Scores of thousands: the running reference has to follow them."""
    for cache in ("bf16", "e4m3"):
        p = make([700, 1500], 4, 2, 128, "bf16", cache, peak=300.0)
        check(idx, p)
    p = make([700], 4, 2, 128, "bf16", "e4m3")
    p["q"] = (p["q"].float() * 2.0 ** 100).bfloat16()  # past fp16's range
    check(idx, p, scale=2.0 ** -104)
    p["q"] = (p["q"].float() * 2.0 ** -210).bfloat16()
    check(idx, p, scale=2.0 ** 100)


@pytest.mark.parametrize("softcap", [0.0, 4.0])
@pytest.mark.parametrize("next_n,k", [(1, 0), (9, 0), (1, 40)])
def test_key_scales_of_either_sign(idx, softcap, next_n, k):
    """A head's negative scale turns its scores around, also under a negative
    softmax scale; a scale of zero makes all of a row's weights equal."""
    p = make([300, 1200, 9], 6, 3, 128, "bf16", "e4m3", next_n=next_n, k=k)
    ks = p["ks"].clone()
    p["ks"] = ks * torch.tensor([1.0, -1.0, 0.0])
    p["k64"] = p["k64"] * np.array([1.0, -1.0, 0.0])[None, :, None, None]
    for scale in (0.1, -0.1):
        check(idx, p, scale=scale, softcap=softcap)


def test_a_key_scale_of_nan_is_not_passed_over(idx):
    p = make([300, 0], 4, 2, 128, "bf16", "e4m3")
    clean, clean_lse = call(idx, p)
    p["ks"] = torch.tensor([float("nan"), p["ks"][1]])
    for softcap in (0.0, 4.0):
        out, lse = call(idx, p, softcap=softcap)
        torch.cuda.synchronize()
        assert torch.isnan(out[0, :2]).all() and torch.isnan(lse[0, :2]).all()
        assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()  # sees nothing
        if not softcap:
            assert torch.equal(out[0, 2:], clean[0, 2:]) and torch.equal(lse[0, 2:], clean_lse[0, 2:])


@pytest.mark.parametrize("n", [300, 5000])
@pytest.mark.parametrize("dtype,cache,group", [("fp16", "fp16", 4), ("fp16", "e4m3", 4),
                                               ("bf16", "e4m3", 16), ("bf16", "bf16", 4)])
def test_few_high_scores_among_many_low_ones(idx, dtype, cache, group, n):
    """Every sixteenth key has a weight near 1 and a value of zero; the result
    is made of the others, whose weights are near 2^-24.  With fp16 operands
    both terms of a weight lie on fp16's smallest grid there: off by half a step
    of 2^-31 of the highest weight."""
    p = make([n], group, 1, 64, dtype, cache, page=16, scales=False)
    pages = len(p["bt"][0])
    q = torch.zeros(p["q"].shape)
    q[:, :, 0] = 16.0
    r = np.random.default_rng(1)
    keys = torch.tensor(-1.0 + r.integers(-4, 5, pages * 16) / 64.0)
    vals = torch.full((pages * 16,), 256.0)
    keys[::16] = 0.0
    vals[::16] = 0.0
    kf, vf = (torch.zeros(p["kc"].shape) for _ in range(2))
    kf[torch.tensor(p["bt"][0].astype(np.int64)), 0, :, 0] = keys.view(-1, 16).float()
    vf[torch.tensor(p["bt"][0].astype(np.int64)), 0] = vals.view(-1, 16, 1).float()
    p["q"], p["kc"], p["vc"] = q.to(p["q"].dtype), kf.to(p["kc"].dtype), vf.to(p["vc"].dtype)
    scale = 1.04
    out, lse = call(idx, p, scale=scale)
    torch.cuda.synchronize()
    ref = su.ref_attention(su.to64(p["q"]), su.to64(p["kc"]), su.to64(p["vc"]), p["bt"], p["lens"],
                           1, float(np.float32(scale)))
    tol, tol_lse = su.attention_tols(*ref, 64, p["dtype"])
    assert 1e-4 < ref[0].min() and ref[0].max() < 1e-3
    if cache != "bf16":
        tol = tol + 15 * 256 * 2.0 ** -32
    assert (np.abs(out.double().cpu().numpy() - ref[0]) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - ref[1]) <= tol_lse).all()


def test_results_do_not_depend_on_the_run(idx):
    p = make([20000, 3000, 1], 8, 2, 128)
    a = call(idx, p)
    for _ in range(5):
        b = call(idx, p)
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_one_workspace_for_different_calls_and_dirty_memory(idx):
    ws = torch.full((max(idx.paged_attention_workspace_bytes(3, 2, 16, 2, 128),
                         idx.paged_attention_workspace_bytes(3, 1, 8, 2, 64)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    for _ in range(2):
        check(idx, make([5000, 0, 700], 16, 2, 128, next_n=2), workspace=ws)
        check(idx, make([9000, 3, 1], 8, 2, 64, page=16), workspace=ws)
        check(idx, make([9000, 3, 1], 16, 2, 128, next_n=2, k=300), workspace=ws)


def test_given_outputs_and_a_short_workspace(idx):
    p = make([300], 4, 2, 128)
    out = torch.full((1, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, 4), 9.0, device="cuda")
    a, b = check(idx, p, out=out, lse=lse)
    assert a is out and b is lse
    with pytest.raises(idx.IdxError) as e:
        call(idx, p, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3


def test_on_another_stream(idx):
    p = make([4000, 50], 8, 2, 128)
    ref = call(idx, p)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call(idx, p)
    s.synchronize()
    assert torch.equal(got[0], ref[0])
    s.wait_stream(torch.cuda.current_stream())
    got = call(idx, p, stream=s)
    s.synchronize()
    # the arguments were made on the current stream, whose work is done by now
    torch.cuda.synchronize()
    assert torch.equal(got[0], ref[0])


def test_graph_replays_read_their_buffers_afresh(idx):
    p = make([3000, 40, 900], 8, 2, 128, page=64)
    q, kc, vc, bt = p["q"].cuda(), p["kc"].cuda(), p["vc"].cuda(), i32(p["bt"])
    lens = i32([1, 1, 1])
    ws = torch.empty(idx.paged_attention_workspace_bytes(3, 1, 8, 2, 128), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 8, device="cuda")
    args = dict(workspace=ws, out=out, lse=lse, return_lse=True)
    idx.paged_attention(q, kc, vc, bt, lens, 1, **args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx.paged_attention(q, kc, vc, bt, lens, 1, **args)
    for now in ([3000, 40, 900], [0, 0, 0], [100, 17, 899], [2999, 1, 0]):
        lens.copy_(i32(now))
        g.replay()
        torch.cuda.synchronize()
        ref = su.ref_attention(su.to64(p["q"]), p["k64"], p["v64"], p["bt"], now, 1,
                               float(np.float32(128 ** -0.5)))
        su.check_attention(out, lse, ref, 128, torch.bfloat16, what=str(now))


def test_strides_of_single_entries_do_not_matter(idx):
    """One request, one kv head, one block: their strides are anything."""
    D = 64
    p = make([16], 1, 1, D, page=16)
    want, _ = call(idx, p)
    q = torch.empty(1, 1, D + 3, dtype=torch.bfloat16, device="cuda")[:, :, :D]
    kc, vc = (torch.empty(16 * D, dtype=torch.bfloat16, device="cuda")
              .as_strided((1, 1, 16, D), (16 * D + 5, 16 * D + 3, D, 1)) for _ in range(2))
    assert q.stride(0) % 8 and kc.stride(0) % 8
    q.copy_(p["q"])
    blk = int(p["bt"][0, 0])
    kc.copy_(p["kc"][blk:blk + 1])
    vc.copy_(p["vc"][blk:blk + 1])
    out = idx.paged_attention(q, kc, vc, i32([[0]]), i32([16]))
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_no_requests(idx):
    kc, vc = idx.new_kv_cache(2, 2, 64)
    out = idx.paged_attention(torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), kc, vc,
                              torch.empty(0, 3, dtype=torch.int32, device="cuda"), i32([]))
    assert out.shape == (0, 4, 64)
