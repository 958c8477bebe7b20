"""Score caps of the paged attention, from far below the scores to far above."""
import numpy as np
import pytest
import torch

import serving_testutil as su
from test_gpu_paged_attention import call, idx, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap", [1e-45, 1e-30, 0.01, 0.5, 4.0, 300.0, 1e3, 1e4, 1e6, 1e8, 1e30,
                                 3.4e38])
@pytest.mark.parametrize("dtype,cache,group,k", [("bf16", "bf16", 4, 0), ("fp16", "fp16", 20, 0),
                                                 ("bf16", "e4m3", 16, 0), ("bf16", "bf16", 2, 90)])
def test_a_cap_of_any_size(idx, cap, dtype, cache, group, k):  # noqa: F811
    """The capped score c tanh(s/c) is as exact, relative to itself, as fp32: a cap
    far above the scores changes nothing, one far below leaves -c, 0 and c.

    Its error: the argument's three roundings, the exponential's and the
    reciprocal's 2^-22 each where tanh is at least a half, and three more
    roundings: 16 half steps of fp32 in all, of a score that the cap makes no
    larger than `smag`.  attention_tols counts dim + 8 of them for the product."""
    p = make([1, 2, 300, 1500], 2 * group, 2, 64, dtype, cache, page=32, k=k)
    c = float(np.float32(cap))
    out, lse = call(idx, p, softcap=c)
    torch.cuda.synchronize()
    ref = su.ref_attention(su.to64(p["q"]), p["k64"], p["v64"], p["bt"], p["lens"], 1,
                           float(np.float32(64 ** -0.5)), c, 0, p["topk"])
    su.check_attention(out, lse, ref, 64 + 16, p["dtype"], what=f"cap {cap}")


def test_a_cap_far_above_the_scores_is_none(idx):  # noqa: F811
    """Within one rounding: the capped score is the score times 1 - (s/c)^2/3."""
    p = make([700, 33], 8, 2, 128, "bf16", "bf16")
    want, want_lse = call(idx, p)
    got, got_lse = call(idx, p, softcap=1e9)
    torch.cuda.synchronize()
    assert (got_lse - want_lse).abs().max() <= 64 * su.U * want_lse.abs().max()
    assert (got.float() - want.float()).abs().max() <= 2 * 2.0 ** -8 * want.float().abs().max()
