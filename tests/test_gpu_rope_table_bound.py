"""Rotary tables against the bound that idx.h states for their entries."""
import numpy as np
import pytest
import torch

import serving_testutil as su
from test_gpu_serving import idx  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(num_pos=200000, rot=128), dict(num_pos=100000, rot=64, base=500000.0),
                                dict(num_pos=60000, rot=256, pos0=2**31 - 60000),
                                dict(num_pos=50000, rot=128, mscale=1.25),
                                dict(num_pos=50000, rot=128, mscale=-0.7071),
                                dict(num_pos=50000, rot=64, scaling="ntk", factor=8.0, mscale=1.9),
                                dict(num_pos=100000, rot=64, scaling="yarn", factor=2.0, orig_len=4096),
                                dict(num_pos=100000, rot=128, scaling="yarn", factor=10.0, orig_len=4096),
                                dict(num_pos=50000, rot=64, scaling="yarn", factor=32.0, orig_len=8192)])
def test_entries_are_within_the_stated_bound(idx, kw):  # noqa: F811
    """1.5 * 2^-24 where mscale is 1, else 3.5 * 2^-24 * |mscale| (mscale's own
    rounding to fp32 and the product's, 2^-24 each), and the angle's error: the
    frequency's fp64 rounding (pow 1 ulp and three operations) at the position."""
    kw = dict(kw)
    n, rot, pos0, mscale = kw.pop("num_pos"), kw.pop("rot"), kw.pop("pos0", 0), kw.pop("mscale", None)
    cos, sin = idx.rope_table(n, rot, pos0=pos0, mscale=mscale, **kw)
    torch.cuda.synchronize()
    m = mscale or 1.0
    if kw.get("scaling") == "yarn" and mscale is None:
        m = 0.1 * np.log(kw["factor"]) + 1.0
    c, s = su.ref_table(pos0, n, rot, mscale=m, **kw)
    tol = (1.5 if m == 1.0 else 3.5 * abs(m)) * su.U + abs(m) * (pos0 + n) * 5 * 2.0 ** -53
    for got, ref in ((cos, c), (sin, s)):
        worst = np.abs(got.cpu().numpy() - ref).max()
        assert worst <= tol, f"{worst / su.U:.3f} half steps of fp32, {tol / su.U:.3f} stated"
