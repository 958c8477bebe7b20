"""Infinities and NaN in positions of the paged cache that some rows of a request
see and others do not."""
import numpy as np
import pytest
import torch

import serving_testutil as su
from test_gpu_paged_attention import call, idx, make  # noqa: F401

pytestmark = pytest.mark.gpu


def check_rows(out, lse, p, rows, window=0):
    """The given rows against the 64-bit form of the values before poison()."""
    ref = su.ref_attention(su.to64(p["q"]), p["k64"], p["v64"], p["bt"], p["lens"], p["next_n"],
                           float(np.float32(p["D"] ** -0.5)), 0.0, window)
    su.check_attention(out[rows], lse[rows], tuple(x[rows] for x in ref), p["D"], p["dtype"])


def poison(p, b, pos, what):
    """A non-finite value row (and key row) at position pos of request b."""
    page = p["kc"].shape[2]
    blk, off = int(p["bt"][b, pos // page]), pos % page
    for name in ("kc", "vc"):
        t = p[name]
        if t.dtype == torch.float8_e4m3fn:
            t.view(torch.uint8)[blk, :, off] = 0x7F
        else:
            t[blk, :, off] = what


@pytest.mark.parametrize("D,dtype,cache,heads,group", [
    (64, "bf16", "bf16", 2, 1), (128, "fp16", "fp16", 2, 2), (128, "bf16", "e4m3", 1, 2),
    (256, "bf16", "bf16", 1, 1), (64, "bf16", "e4m3", 3, 4), (128, "bf16", "bf16", 2, 8),
    (64, "fp16", "fp16", 1, 16), (256, "fp16", "e4m3", 2, 9), (128, "bf16", "e4m3", 1, 24)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("next_n,window", [(2, 0), (5, 0), (3, 40)])
def test_a_position_that_is_not_finite_reaches_the_rows_that_see_it_alone(
        idx, D, dtype, cache, heads, group, what, next_n, window):  # noqa: F811
    """The last new token's key and value (seen by the last row alone) and, with a
    window, the first position (gone from the last row's sight)."""
    lens = [200, next_n, 64, 65, 129]
    p = make(lens, heads * group, heads, D, dtype, cache, page=16, next_n=next_n)
    hit = np.zeros((len(lens), next_n), bool)
    for b, n in enumerate(lens):
        for pos in [n - 1] + ([n - next_n - window + 1] if window and n > window + next_n else []):
            poison(p, b, pos, what)
            for j in range(next_n):
                end = n - next_n + 1 + j
                hit[b, j] |= pos < end and (not window or pos >= end - window)
    out, lse = call(idx, p, window=window)
    torch.cuda.synchronize()
    hit = hit.reshape(-1)
    assert hit.any() and not hit.all()
    check_rows(out, lse, p, ~hit, window)
    assert not torch.isfinite(out[torch.from_numpy(hit).cuda()]).all(-1).any()


@pytest.mark.parametrize("D,dtype,cache,group", [(128, "bf16", "bf16", 3), (64, "bf16", "e4m3", 3),
                                                 (128, "fp16", "fp16", 12), (256, "bf16", "e4m3", 6)])
def test_a_value_that_is_not_finite_stays_in_its_dimension(idx, D, dtype, cache, group):  # noqa: F811
    """One value of the last new token: the last row's dimension alone."""
    p = make([77, 500], group, 1, D, dtype, cache, page=16, next_n=2)
    clean, clean_lse = call(idx, p)
    for b, n in enumerate(p["lens"]):
        blk, off = int(p["bt"][b, (n - 1) // 16]), (n - 1) % 16
        for d in (0, 5, 17, 46, D - 1):
            if cache == "e4m3":
                p["vc"].view(torch.uint8)[blk, 0, off, d] = 0xFF
            else:
                p["vc"][blk, 0, off, d] = float("nan")
    out, lse = call(idx, p)
    torch.cuda.synchronize()
    assert torch.equal(lse, clean_lse)
    off = torch.zeros_like(out, dtype=torch.bool)
    off[1::2][:, :, [0, 5, 17, 46, D - 1]] = True
    assert torch.equal(torch.isnan(out), off) and torch.equal(out[~off], clean[~off])


def test_a_split_call_keeps_masked_values_out_too(idx):  # noqa: F811
    p = make([20000, 9000], 4, 2, 64, page=16, next_n=2)
    for b, n in enumerate(p["lens"]):
        poison(p, b, n - 1, float("nan"))
    out, lse = call(idx, p)
    torch.cuda.synchronize()
    check_rows(out, lse, p, np.array([True, False, True, False]))
    assert torch.isnan(out[1::2]).all()
