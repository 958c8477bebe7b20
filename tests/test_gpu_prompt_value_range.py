"""Prompt attention in bf16 at both ends of the type's range: outputs are finite whatever the
length where values are at most 2^127, and small values keep what the type holds of them."""
import pytest
import torch

import prompt_testutil as pu
from test_gpu_prompt_attention import make, run, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def idx():
    from sparse_attention_indexer_quant_gb300 import binding
    binding.check_device(torch.cuda.current_device())
    return binding


def check(idx, q, k, v, lens, keys, **kw):
    """pu.prompt_tols, half of bf16's smallest step, and the sums' own steps: they are kept in fp32
    at a scale where all weights sum to 2^-15 or more, so that a step of 2^-149 for every 16 keys
    (two for a product that truncates) is 2^-137 a key."""
    out, lse = run(idx, q, k, v, lens, keys, scale=1.0, **kw)
    ref = pu.ref_prompt(q, k, v, starts(lens), starts(keys), 1.0, **kw)
    tol, tol_lse = pu.prompt_tols(ref, q.shape[2], torch.bfloat16)
    tol = tol + 2.0 ** -134 + ref[4][:, None, None] * 2.0 ** -137
    assert torch.isfinite(out).all()
    assert ((out.double() - ref[0]).abs() <= tol).all()
    live = torch.isfinite(ref[1])
    assert torch.equal(torch.isneginf(lse), ~live)
    assert ((lse.double() - ref[1]).abs()[live] <= tol_lse[live]).all()


def climbing(n, L, Hq, Hkv, D, low, step, power):
    """Scores of 0 at the first `low` keys, then `step`; positive values of 2^(power-1) to 2^power."""
    g = torch.Generator(device="cuda").manual_seed(L + D)
    q, k = torch.zeros(n, Hq, D, device="cuda"), torch.zeros(L, Hkv, D, device="cuda")
    q[..., 0], k[low:, :, 0] = 1.0, step
    v = (0.5 + 0.499 * torch.rand(L, Hkv, D, device="cuda", generator=g)) * 2.0 ** power
    return q.bfloat16(), k.bfloat16(), v.bfloat16()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("power", [127, 110, 100])
@pytest.mark.parametrize("n,L,Hq,Hkv", [(40, 700, 4, 1),   # keys of one CTA
                                        (3, 30000, 4, 1),  # shared out among a cluster
                                        (60, 5000, 80, 80)])
def test_large_values_of_many_keys(idx, D, power, n, L, Hq, Hkv):
    """6.5 is 9.4 in log2: 64 such weights sum to less than 2^16 of the first ones."""
    check(idx, *climbing(n, L, Hq, Hkv, D, 128, 6.5, power), [n], [L])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_values_of_equal_keys(idx, D):
    check(idx, *climbing(5, 9000, 2, 1, D, 0, 0.0, 127), [5], [9000])
    check(idx, *climbing(150, 400, 2, 1, D, 0, 0.0, 127), [150], [400])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("power", [-100, -118, -126])
@pytest.mark.parametrize("step", [0.0, 6.5])
def test_small_values(idx, D, power, step):
    check(idx, *climbing(40, 700, 4, 1, D, 128, step, power), [40], [700])
    check(idx, *climbing(3, 20000, 4, 1, D, 128, step, power), [3], [20000])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("power", [-110, 120])
def test_random_scores(idx, D, power):
    lens, keys = [70, 3, 40], [3000, 3, 500]
    q, k, v = make(lens, keys, 4, 2, D, "bf16", peak=2 * D ** -0.5)
    check(idx, q, k, v * 2.0 ** power, lens, keys)
    check(idx, q, k, v * 2.0 ** power, lens, keys, window=300)
