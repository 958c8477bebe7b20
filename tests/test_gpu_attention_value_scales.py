"""Value scales of an E4M3 cache that are not finite."""
import pytest
import torch

from test_gpu_paged_attention import call, idx, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("lens,k", [([0, 300, 0, 7], 0), ([0, 40000], 0), ([0, 300, 9], 40)])
def test_a_value_scale_that_is_not_finite_leaves_empty_rows_zero(idx, bad, lens, k):  # noqa: F811
    p = make(lens, 4, 2, 128, "bf16", "e4m3", k=k)
    p["vs"] = torch.tensor([bad, 0.5])
    out, lse = call(idx, p)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all() and torch.isneginf(lse[b]).all()
        else:
            assert not torch.isfinite(out[b, :2]).any() and torch.isfinite(out[b, 2:]).all()
