"""Attention over a 4-bit cache at both ends of its values' range: blocks from scale byte 0
(2^-127) up to values of 2^54, alone and side by side, whole, split and selected."""
import numpy as np
import pytest
import torch

import mxfp4_testutil as mx
import serving_testutil as su
from test_gpu_kv4 import attend, make

pytestmark = pytest.mark.gpu

SMALLEST_HALF_STEP = 2.0 ** -134  # of bf16


@pytest.fixture(scope="module")
def idx():
    from sparse_attention_indexer_quant_gb300 import binding
    binding.check_device(torch.cuda.current_device())
    return binding


def scaled(p, power):
    """The cache's values times 2^power, an array that broadcasts to [blocks, heads, page, D / 32]."""
    codes, scales = mx.from_pages(p["vc"])
    new = np.where(scales == 255, 255, scales.astype(int) + power)
    assert new.min() >= 0 and new.max() <= 255
    p["vc"] = mx.to_pages(codes, new.astype(np.uint8))
    power = np.broadcast_to(power, scales.shape)
    p["v64"] = p["v64"] * 2.0 ** np.repeat(power, 32, -1).astype(np.float64)


def check(idx, p, **kw):
    """su.check_attention's tolerance, and half of bf16's smallest step."""
    out, lse = attend(idx, p, **kw)
    ref = su.ref_attention(su.to64(p["q"]), p["k64"], p["v64"], p["bt"], p["lens"], p["next_n"], p["D"] ** -0.5,
                           topk=p["topk"], **kw)
    tol, tol_lse = su.attention_tols(*ref, p["D"], p["dtype"])
    assert (np.abs(su.to64(out.cpu()) - ref[0]) <= tol + SMALLEST_HALF_STEP).all()
    assert (np.abs(lse.double().cpu().numpy() - ref[1]) <= tol_lse).all()


# (values of N(0, 1) have scale bytes from 124 on, and are below 2^3)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [4, 16])
@pytest.mark.parametrize("power", [-124, -120, -100, -88, -78, -70, 51])
def test_values_of_one_size(idx, D, group, power):
    p = make([300, 9000], 2 * group, 2, D)
    scaled(p, power)
    check(idx, p)


@pytest.mark.parametrize("group", [4, 40])
@pytest.mark.parametrize("power", [-120, 51])
def test_selected_values(idx, group, power):
    p = make([700, 90], 2 * group, 2, 128, k=300, page=32)
    scaled(p, power)
    check(idx, p)


@pytest.mark.parametrize("group", [4, 16])
def test_large_and_small_values_side_by_side(idx, group):
    """Neighbouring blocks of dimensions, and heads, at the two ends."""
    p = make([300, 5000], 2 * group, 2, 128)
    power = np.array([51, -120, -60, 0])[None, None, None, :] * np.array([1, -1])[None, :, None, None]
    scaled(p, np.clip(power, -120, 51))
    check(idx, p)


@pytest.mark.parametrize("group", [4, 16])
@pytest.mark.parametrize("first", [True, False])
def test_large_values_of_keys_that_hardly_count(idx, group, first):
    """Keys whose weight is 2^-120 of the others' hold the large values, the others the small ones: the
    sums are those of the others to the large values' share."""
    D, L = 128, 4000
    p = make([L], 2 * group, 2, D)
    at = np.arange(L)
    low = at < 1000 if first else at >= 3000
    codes, scales = mx.from_pages(p["kc"])
    pages = p["bt"][0][at // 64], at % 64
    # every key is its first dimension alone: 6 there, or 0
    codes[pages[0], :, pages[1]] = 0
    scales[pages[0], :, pages[1]] = 127
    codes[pages[0][~low], :, pages[1][~low], 0] = 7
    p["kc"] = mx.to_pages(codes, scales)
    p["k64"][pages[0], :, pages[1]] = mx.decode64(codes, np.where(scales == 255, 0, scales))[pages[0], :, pages[1]]
    p["q"] = torch.zeros_like(p["q"])
    p["q"][..., 0] = 120 * float(np.log(2)) / 6 * D ** 0.5
    power = np.zeros((scales.shape[0], 1, scales.shape[2], 1), int)
    power[pages[0], 0, pages[1]] = np.where(low, 40, -70)[:, None]
    scaled(p, power)
    check(idx, p)
