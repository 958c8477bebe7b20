"""The 4-bit insert over the whole range of keys, weights and eps: codes and scales are those of
64-bit arithmetic where fp32's squares, factors or products would overflow or lose bits; and a
stored token changes its own bytes alone."""
import numpy as np
import pytest
import torch

import mxfp4_testutil as mx
import serving_testutil as su

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def idx():
    from sparse_attention_indexer_quant_gb300 import binding
    binding.check_device(torch.cuda.current_device())
    return binding


def insert_and_check(idx, k, w, eps, rot, interleaved, angles=6.3):
    N, Hkv, D = k.shape
    page = 32
    g = torch.Generator().manual_seed(D)
    angle = angles * torch.rand(500, max(1, rot // 2), generator=g)
    cos, sin = torch.cos(angle), torch.sin(angle)
    pos = torch.randint(0, 500, (N,), generator=g)
    kc, vc = idx.new_kv_cache(N // page + 1, Hkv, D, "mxfp4", page)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    tables = (pos.int().cuda(), cos.cuda(), sin.cuda(), rot) if rot else (None, None, None, 0)
    idx.qk_norm_rope_insert(k.cuda(), k.cuda(), k.cuda(), cu(w), cu(w), eps, *tables, torch.arange(N, device="cuda"),
                            kc, vc, interleaved=interleaved)
    x, _ = su.ref_turned(k.double().numpy(), None if w is None else w.double().numpy(), float(np.float32(eps)),
                         cos[pos].double().numpy(), sin[pos].double().numpy(), rot, interleaved)
    codes, scales = mx.from_pages(kc.cpu())
    at = np.arange(N)
    c, s = codes[at // page, :, at % page], scales[at // page, :, at % page]
    wc, ws = mx.encode64(x)
    assert (s == ws).all()
    # (a zero's sign is not a value)
    assert (np.where(c == 8, 0, c) == np.where(wc == 8, 0, wc)).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("power,eps", [(65, 1e-6), (70, 0.0), (120, 1e-6), (-70, 0.0), (-75, 1e-6), (-120, 0.0),
                                       (-60, 1e-30)])
def test_normed_keys_of_any_size(idx, D, interleaved, power, eps):
    g = torch.Generator().manual_seed(D + power)
    w = 1 + 0.2 * torch.randn(D, generator=g)
    for N in (60, 1500):
        k = (torch.randn(N, 2, D, generator=g) * 2.0 ** power).bfloat16()
        insert_and_check(idx, k, w, eps, D // 2, interleaved)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("power", [61, 64, 70, 120])
def test_large_positive_keys(idx, D, power):
    """The sum of squares is infinite in fp32; no value's sign tells."""
    g = torch.Generator().manual_seed(D + power)
    w = 1 + 0.2 * torch.rand(D, generator=g)
    for N in (60, 1500):
        k = ((0.1 + torch.rand(N, 2, D, generator=g)) * 2.0 ** power).bfloat16()
        insert_and_check(idx, k, w, 1e-6, 0, False)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("power,weight,eps", [(0, -60, 1e-6), (0, 60, 1e-6), (100, -110, 0.0), (-60, -60, 1e-6),
                                              (60, -120, 0.0), (-100, 100, 1e-6)])
def test_weights_of_any_size(idx, interleaved, power, weight, eps):
    g = torch.Generator().manual_seed(weight)
    k = (torch.randn(1500, 2, 128, generator=g) * 2.0 ** power).bfloat16()
    insert_and_check(idx, k, (1 + 0.2 * torch.randn(128, generator=g)) * 2.0 ** weight, eps, 128, interleaved)


@pytest.mark.parametrize("dtype,power", [(torch.bfloat16, -124), (torch.bfloat16, -116), (torch.bfloat16, 120),
                                         (torch.float16, -14)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_turned_keys_of_any_size(idx, dtype, power, interleaved):
    g = torch.Generator().manual_seed(3)
    k = (torch.randn(1500, 2, 64, generator=g) * 2.0 ** power).to(dtype)
    insert_and_check(idx, k, None, 0.0, 64, interleaved)
    insert_and_check(idx, k, None, 0.0, 64, interleaved, angles=2.0 ** -30)  # sines that make products small


def test_zeros_among_normed_keys(idx):
    g = torch.Generator().manual_seed(5)
    k = torch.randn(300, 2, 128, generator=g).bfloat16()
    k[::3], k[1::3, :, 32:64], k[2::3, :, ::2] = 0, 0, 0
    w = torch.randn(128, generator=g)
    w[64:80] = 0
    for interleaved in (False, True):
        insert_and_check(idx, k, w, 1e-6, 64, interleaved)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_token_changes_its_own_bytes_alone(idx, D):
    """Slots outside the cache are counted and store nothing, -1 stores nothing; the token that has a
    slot gets its codes and scales there."""
    g = torch.Generator().manual_seed(D)
    page, blocks, Hkv = 16, 2, 3
    fill = torch.full((blocks, Hkv, page, D * 17 // 32), 0x5A, dtype=torch.uint8)
    kc, vc = fill.cuda(), fill.cuda()
    k, v = torch.randn(2, 5, Hkv, D, generator=g).bfloat16()
    errs = idx.new_errors()
    idx.qk_norm_rope_insert(k.cuda(), k.cuda(), v.cuda(), None, None, 0.0, None, None, None, 0,
                            torch.tensor([32, -7, 5, -1, 1 << 40], device="cuda"), kc, vc, errors=errs)
    assert errs.tolist() == [3, 0]
    for cache, x in ((kc, k), (vc, v)):
        codes, scales = mx.from_pages(fill)
        scales = scales.copy()
        codes[0, :, 5], scales[0, :, 5] = mx.encode64(x[2].double().numpy())
        assert torch.equal(cache.cpu(), mx.to_pages(codes, scales))
