"""Every kernel of the paged attention, and every way in which a split call is cut,
each reached by a shape that is checked to reach it: values against the 64-bit
form, runs against each other, dirty and shared workspaces, graph replays."""
import numpy as np
import pytest
import torch

import attention_forms as af
import serving_testutil as su

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def idx():
    from sparse_attention_indexer_quant_gb300 import binding
    binding.check_device(torch.cuda.current_device())
    return binding


def run(idx, p, softcap=0.0, window=0, **more):
    errs = idx.new_errors()
    args, kw = p.on_gpu()
    out, lse = idx.paged_attention(*args, **kw, softcap=softcap, window=window, errors=errs, **more)
    torch.cuda.synchronize()
    assert errs.cpu().tolist() == [0, 0]
    return out, lse


def check(idx, p, softcap=0.0, window=0, ref=None, **more):
    out, lse = run(idx, p, softcap, window, **more)
    ref = p.reference(float(np.float32(softcap)), window) if ref is None else ref
    su.check_attention(out, lse, ref, p.D, p.dtype, softcap)
    return out, lse


@pytest.mark.parametrize("D,cache,tiles,sights,warps", af.FORMS)
def test_every_kernel(idx, D, cache, tiles, sights, warps):
    args = af.shape_for(idx, D, cache, tiles, sights, warps)
    if args is None:
        pytest.skip("no shape for this number of SMs")
    p = af.Problem(**args)
    form = idx.paged_attention_form(*p.form_args)
    assert (0 if form.split else form.warps) == warps
    assert form.rows * form.row_tiles >= p.q.shape[1] // p.heads * p.next_n
    check(idx, p)
    check(idx, p, softcap=20.0)


def problem(idx, name):
    way, args = af.WAYS[name]
    p = af.Problem(**args)
    if af.way_of(idx, p) != way:
        pytest.skip("cut differently for this number of SMs")
    return p


@pytest.mark.parametrize("name", list(af.WAYS))
def test_every_way_of_cutting(idx, name):
    """The result, and the same bytes from run to run, also out of a workspace that
    holds all ones, a small number everywhere or the last call's state."""
    p = problem(idx, name)
    first = check(idx, p)
    size = idx.paged_attention_workspace_bytes(*p.form_args[:5])
    for fill in (0xFF, 0x01, None, None, None):
        if fill is not None:
            ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        again = run(idx, p, workspace=ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_calls_cut_in_different_ways_share_a_workspace(idx):
    names = ["claimed, 320 requests", "equal, ragged", "claimed, few long", "pieces, ragged",
             "claimed, selections"]
    ps = [problem(idx, n) for n in names]
    want = [run(idx, p) for p in ps]
    ws = torch.full((max(idx.paged_attention_workspace_bytes(*p.form_args[:5]) for p in ps),), 0xA5,
                    dtype=torch.uint8, device="cuda")
    for i in (0, 1, 0, 2, 3, 2, 4, 0, 4, 4, 1, 2):
        got = run(idx, ps[i], workspace=ws)
        assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1]), names[i]


@pytest.mark.parametrize("name", ["claimed, 320 requests", "claimed, few long", "equal, ragged",
                                  "pieces, ragged"])
def test_graph_replays_of_split_calls(idx, name):
    """Replays use the captured call's generation over and over, with other lengths
    each time, and with another call in the same workspace between them."""
    p = problem(idx, name)
    (q, k, v, bt, lens, next_n), kw = p.on_gpu()
    ws = torch.full((idx.paged_attention_workspace_bytes(*p.form_args[:5]),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    kw.update(workspace=ws, out=out, lse=lse)
    idx.paged_attention(q, k, v, bt, lens, next_n, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx.paged_attention(q, k, v, bt, lens, next_n, **kw)
    r = np.random.default_rng(0)
    fewer = [0 if r.random() < 0.2 else int(n * r.uniform(0.7, 1)) for n in p.lens]
    refs = {}
    for what, now in (("all", p.lens), ("all", p.lens), ("fewer", fewer), ("none", [0] * len(fewer)),
                      ("fewer", fewer), ("all", p.lens)):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        if what not in refs:
            refs[what] = p.reference(lens=now)
        su.check_attention(out, lse, refs[what], p.D, p.dtype, what=what)
        run(idx, p, workspace=ws)
    if name.startswith("claimed"):
        assert af.way_of(idx, p, fewer) == "claimed"


@pytest.mark.parametrize("next_n", [2, 3])
def test_a_claimed_split_with_windows_and_caps(idx, next_n):
    p = af.Problem(af.ragged(5, 320, 300, (0, 300)), 16, 1, 64, next_n=next_n, page=16, room=40000)
    assert af.way_of(idx, p) == "claimed"
    check(idx, p, softcap=30.0)
    check(idx, p, window=77)  # its room is the window's: shared out differently
