"""How attention calls are shared out, from their sizes: the query, and that the
shapes the GPU tests use reach every kernel and every way of cutting."""
import pytest
import torch

import attention_forms as af

SMS = 152


@pytest.fixture(scope="module")
def idx():
    from sparse_attention_indexer_quant_gb300 import binding
    return binding


def test_form_of_known_calls(idx):
    f = idx.paged_attention_form(64, 1, 32, 8, 128, max_blocks=512, sms=SMS)  # a long batch
    assert f.split and f.rows == 4 and f.row_tiles == 1 and f.places == 2 * SMS
    f = idx.paged_attention_form(64, 1, 32, 8, 128, max_blocks=512, topk=2048, sms=SMS)
    assert not f.split and f.warps == 4 and f.places == 2 * SMS * 2
    f = idx.paged_attention_form(1, 1, 32, 8, 128, max_blocks=3, sms=SMS)  # one short request
    assert not f.split and f.warps == 8
    f = idx.paged_attention_form(1, 16, 64, 1, 256, max_blocks=4, sms=SMS)  # 1024 rows by sixteens
    assert f.rows == 16 and f.row_tiles == 64


@pytest.mark.parametrize("bad", [dict(next_n=0), dict(Hq=7), dict(Hkv=0), dict(head_dim=96),
                                 dict(page_size=48), dict(max_blocks=0), dict(topk=-1), dict(window=-1),
                                 dict(topk=4, window=4), dict(sms=0), dict(sms=5000), dict(B=-1)])
def test_form_refuses(idx, bad):
    a = dict(B=1, next_n=1, Hq=8, Hkv=8, head_dim=128, page_size=64, max_blocks=4, topk=0, window=0, sms=SMS)
    idx.paged_attention_form(**a)
    with pytest.raises(idx.IdxError):
        idx.paged_attention_form(**{**a, **bad})
    with pytest.raises(TypeError):
        idx.paged_attention_form(**a, cache_dtype=torch.float32)
    assert idx.lib.idx_paged_attention_form(1, 1, 8, 8, 128, 0, 64, 4, 0, 0, SMS, None) == 1


@pytest.mark.parametrize("D,cache,tiles,sights,warps", af.FORMS)
def test_a_shape_reaches_every_kernel(idx, D, cache, tiles, sights, warps):
    assert af.shape_for(idx, D, cache, tiles, sights, warps, SMS)


@pytest.mark.parametrize("name", list(af.WAYS))
def test_shapes_are_cut_as_named(idx, name):
    way, args = af.WAYS[name]
    a = dict(args)
    page, topk = a.get("page", 64), a.get("topk", 0)
    mb = -(-max(max(a["lens"]), a.get("room", 0)) // page)
    f = idx.paged_attention_form(len(a["lens"]), a.get("next_n", 1), a["heads"] * a["group"], a["heads"], a["D"],
                                 af.TYPES[a.get("cache", "bf16")], page, mb, topk, sms=SMS)
    assert f.split
    assert af.cut(f, a["lens"], a.get("next_n", 1), a["heads"], topk).way == way
