"""The step plan's arrays may not overlap where one of them is written, but for
lengths that are advanced in place."""
import numpy as np
import pytest
import torch

import serving_testutil as su
from test_serving_host import INVALID, plan_args

IN = dict(cached=0x10000, new=0x20000, free=0x30000, head=0x40000)
OUT = dict(ctx=0x50000, start=0x60000, slots=0x70000, pos=0x80000, seq=0x90000, head_out=0xA0000,
           bt=0xB0000)
SIZE = dict(cached=4000, new=4000, free=4000, head=4, ctx=4000, start=4004, slots=8000, pos=4000,
            seq=4000, head_out=4, bt=16000)


def refuse(**kw):
    """Addresses that are never read: the call is refused before anything runs."""
    from sparse_attention_indexer_quant_gb300 import binding as idx
    args = plan_args(**{**dict(B=1000, num_free=1000, num_tokens=1000, max_blocks=4), **IN, **OUT, **kw})
    assert idx.lib.idx_plan_step(*args) == INVALID
    assert b"overlaps" in idx.lib.idx_last_error_detail()


@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("other", list(IN) + list(OUT))
def test_overlaps_are_refused(out, other):
    if out == other:
        return
    at = {**IN, **OUT}[other]
    if (out, other) != ("ctx", "cached"):
        refuse(**{out: at})
    if SIZE[other] > 8:
        refuse(**{out: at + SIZE[other] - 8 if out == "slots" else at + SIZE[other] - 4})
    if SIZE[out] > 8:
        refuse(**{out: at - SIZE[out] + (8 if out == "slots" else 4)})


def test_lengths_advanced_in_place_overlap_nothing_else():
    refuse(cached=OUT["ctx"], new=OUT["ctx"])
    refuse(cached=OUT["ctx"], new=OUT["ctx"] + 400)
    refuse(cached=OUT["ctx"], free=OUT["ctx"] + 400)


@pytest.mark.gpu
@pytest.mark.parametrize("B,page,hi", [(1, 64, 5), (7, 16, 700), (256, 64, 1), (1025, 16, 9),
                                       (3000, 32, 3)])
def test_lengths_advance_in_place(B, page, hi):
    from sparse_attention_indexer_quant_gb300 import binding as idx
    r = np.random.default_rng(B)
    steps = [r.integers(0, hi + 1, B) for _ in range(4)]
    most = [int(s.sum()) for s in steps]
    num_blocks = sum(-(-int(x) // page) for x in sum(steps)) + 5
    mb = max(-(-int(x) // page) for x in sum(steps)) + 2
    free = r.permutation(num_blocks).astype(np.int32)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    lens, bt, dfree, head = i32(np.zeros(B)), torch.full((B, mb), -3, dtype=torch.int32, device="cuda"), i32(free), i32([0])
    ref_lens, ref_bt, ref_head = np.zeros(B, np.int64), bt.cpu().numpy(), 0
    errs = idx.new_errors()
    for new, n in zip(steps, most):
        empty = idx.plan_step(lens, i32(new), bt.clone(), dfree, head, n + 3, num_blocks, page_size=page)
        out = empty._replace(context_lens=lens)
        p = idx.plan_step(lens, i32(new), bt, dfree, head, n + 3, num_blocks, page_size=page, out=out,
                          errors=errs)
        assert p.context_lens is lens
        torch.cuda.synchronize()
        want = su.ref_plan(ref_lens, new, ref_bt, free, ref_head, n + 3, num_blocks, page)
        for got, ref, name in zip(p, want[:5], p._fields):
            assert np.array_equal(got.cpu().numpy(), ref), name
        assert np.array_equal(bt.cpu().numpy(), want[6])
        assert all(torch.equal(a, b) for a, b in zip(p, empty))
        ref_lens, ref_bt, ref_head = want[0].astype(np.int64), want[6], want[5]
        head = p.pool_head.clone()
    assert errs.cpu().tolist() == [0, 0]


@pytest.mark.gpu
def test_a_chain_in_place_in_a_graph():
    from sparse_attention_indexer_quant_gb300 import binding as idx
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    lens, new, bt = i32([5, 0, 40]), i32([200, 150, 100]), i32(np.zeros((3, 80)))
    bt[0, 0], bt[2, :3] = 1, i32([2, 3, 4])
    free, head = i32(np.arange(10, 200)), i32([0])
    plan = idx.plan_step(lens, new, bt.clone(), free, head, 450, 300, page_size=16)
    plan = plan._replace(context_lens=lens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx.plan_step(lens, new, bt, free, head, 450, 300, page_size=16, out=plan)
        head.copy_(plan.pool_head)
    ref_lens, ref_bt, ref_head = lens.cpu().numpy(), bt.cpu().numpy(), 0
    for _ in range(6):
        g.replay()
        torch.cuda.synchronize()
        want = su.ref_plan(ref_lens, [200, 150, 100], ref_bt, np.arange(10, 200), ref_head, 450, 300, 16)
        ref_lens, ref_bt, ref_head = want[0], want[6], want[5]
        assert np.array_equal(lens.cpu().numpy(), ref_lens)
        assert np.array_equal(plan.slot_mapping.cpu().numpy(), want[2])
        assert np.array_equal(bt.cpu().numpy(), ref_bt)
