"""Host side of the serving operators, without a GPU: argument refusals through
the C ABI and the binding, workspace sizes, and pins of the plain forms the GPU
tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

from sparse_attention_indexer_quant_gb300 import binding as idx
import serving_testutil as su

INVALID, TOO_SMALL = 1, 3


def kv(**kw):
    a = dict(k=1 << 12, v=1 << 12, k_scale=None, v_scale=None, num_blocks=8, k_block_stride=65536,
             k_head_stride=8192, k_token_stride=128, v_block_stride=65536, v_head_stride=8192,
             v_token_stride=128, page_size=64, heads=8, head_dim=128, dtype=0)
    a.update(kw)
    return idx.KvCacheStruct(*[a[n] for n, _ in idx.KvCacheStruct._fields_])


BAD_KV = [dict(page_size=48), dict(page_size=256), dict(head_dim=96), dict(head_dim=0),
          dict(heads=0), dict(heads=2000), dict(num_blocks=0), dict(num_blocks=1 << 40),
          dict(num_blocks=1 << 25), dict(k_block_stride=-8), dict(v_token_stride=100),
          dict(k_head_stride=1 << 60), dict(dtype=1), dict(dtype=5), dict(k_scale=4096)]


def plan_args(**kw):
    a = dict(cached=None, new=None, B=0, bt=None, max_blocks=4, free=None, num_free=0, head=None,
             head_out=None, num_blocks=8, page=64, ctx=None, start=None, slots=None, pos=None,
             seq=None, num_tokens=0, errors=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [dict(B=-1), dict(B=70000), dict(max_blocks=0),
                                 dict(max_blocks=1 << 25), dict(num_free=-1), dict(page=48),
                                 dict(page=8), dict(num_blocks=0), dict(num_blocks=1 << 33),
                                 dict(num_tokens=-1), dict(num_tokens=1 << 33)])
def test_plan_step_refuses(bad):
    assert idx.lib.idx_plan_step(*plan_args(**bad)) == INVALID
    assert idx.lib.idx_last_error_detail()


def table_args(**kw):
    a = dict(pos0=0, num_pos=4, rot=64, base=1e4, scaling=0, factor=1.0, orig=0.0, fast=32.0,
             slow=1.0, mscale=1.0, cos=None, sin=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [dict(pos0=-1), dict(num_pos=-1), dict(pos0=1 << 31, num_pos=1),
                                 dict(rot=0), dict(rot=63), dict(rot=258), dict(base=1.0),
                                 dict(base=float("inf")), dict(base=float("nan")),
                                 dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.0),
                                 dict(scaling=1, factor=float("nan")), dict(scaling=2, rot=2),
                                 dict(scaling=3, orig=0.0), dict(scaling=3, orig=4096.0, slow=0.0),
                                 dict(scaling=3, orig=4096.0, fast=0.5), dict(mscale=float("inf"))])
def test_rope_table_refuses(bad):
    assert idx.lib.idx_rope_table(*table_args(**bad)) == INVALID
    assert idx.lib.idx_last_error_detail()


def insert_args(kvs, **kw):
    a = dict(q=None, q_ts=1024, q_hs=128, k=None, k_ts=1024, k_hs=128, v=None, v_ts=1024,
             v_hs=128, N=0, Hq=8, dtype=0, qw=None, kw=None, eps=1e-6, pos=None, cos=None,
             sin=None, num_pos=16, rot=64, inter=0, slots=None, q_out=None,
             kv=ctypes.byref(kvs), errors=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", BAD_KV)
def test_insert_refuses_caches(bad):
    assert idx.lib.idx_qk_norm_rope_insert(*insert_args(kv(**bad))) == INVALID
    assert idx.lib.idx_last_error_detail()


@pytest.mark.parametrize("bad", [dict(N=-1), dict(N=1 << 30), dict(Hq=0), dict(Hq=5000),
                                 dict(dtype=2), dict(dtype=7), dict(rot=-2), dict(rot=130),
                                 dict(rot=7, inter=1), dict(rot=24), dict(num_pos=-1),
                                 dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                                 dict(q_ts=100), dict(k_hs=-8), dict(v_ts=1 << 60), dict(kv=None),
                                 dict(N=1 << 26, Hq=4096)])
def test_insert_refuses(bad):
    assert idx.lib.idx_qk_norm_rope_insert(*insert_args(kv(), **bad)) == INVALID
    assert idx.lib.idx_last_error_detail()


def attn_args(kvs, **kw):
    a = dict(q=None, q_ts=1024, q_hs=128, dtype=0, B=0, next_n=1, Hq=8, kv=ctypes.byref(kvs),
             bt=None, max_blocks=4, lens=None, topk_idx=None, topk=0, scale=1.0, softcap=0.0,
             window=0, out=None, lse=None, ws=None, ws_bytes=0, errors=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", BAD_KV)
def test_attention_refuses_caches(bad):
    assert idx.lib.idx_paged_attention(*attn_args(kv(**bad))) == INVALID


@pytest.mark.parametrize("bad", [dict(dtype=2), dict(B=-1), dict(B=70000), dict(next_n=0),
                                 dict(next_n=17), dict(Hq=0), dict(Hq=12), dict(Hq=4104),
                                 dict(B=65535, next_n=16, Hq=32), dict(q_ts=12), dict(q_hs=-8),
                                 dict(max_blocks=0), dict(max_blocks=1 << 26),
                                 dict(scale=float("nan")), dict(scale=float("inf")),
                                 dict(softcap=-1.0), dict(softcap=float("nan")),
                                 dict(window=-1), dict(kv=None),
                                 dict(topk_idx=4096, topk=0), dict(topk_idx=4096, topk=1 << 21),
                                 dict(topk_idx=4096, topk=4, window=7)])
def test_attention_refuses(bad):
    assert idx.lib.idx_paged_attention(*attn_args(kv(), **bad)) == INVALID
    assert idx.lib.idx_last_error_detail()


def test_attention_workspace_is_host_only():
    one = idx.paged_attention_workspace_bytes(1, 1, 8, 8, 64)
    big = idx.paged_attention_workspace_bytes(64, 2, 64, 8, 128)
    assert 0 < one <= big
    # the same for every batch up to the items' descriptors
    assert idx.paged_attention_workspace_bytes(64, 1, 32, 8, 128) - \
        idx.paged_attention_workspace_bytes(1, 1, 32, 8, 128) <= 64 * 8 * 8 + 256
    assert idx.paged_attention_workspace_bytes(1, 1, 7, 2, 128) == 0
    assert idx.paged_attention_workspace_bytes(1, 0, 8, 8, 128) == 0


def test_binding_refuses_what_the_library_cannot_see():
    c = torch.zeros(4, 2, 64, 128, dtype=torch.bfloat16)
    i32 = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        idx.paged_attention(c[0], c, c, i32, i32)
    with pytest.raises(TypeError):
        idx.paged_attention(c[0], c.float(), c.float(), i32, i32)
    with pytest.raises(TypeError):
        idx.paged_attention(c[0], c, c.half(), i32, i32)
    with pytest.raises(ValueError, match="CUDA"):
        idx.plan_step(i32, i32, i32[None], i32, i32, 1, 4)
    with pytest.raises(TypeError):
        idx.plan_step([1], i32, i32[None], i32, i32, 1, 4)
    with pytest.raises(ValueError, match="scaling"):
        idx.rope_table(4, 8, scaling="other")
    with pytest.raises(ValueError, match="CUDA"):
        idx.qk_norm_rope_insert(c[0], c[0], c[0], None, None, 0.0, i32, None, None, 0,
                                i32.long(), c, c)


# ------------------------------------------------------------------ the plain forms, by hand

def test_ref_plan_by_hand():
    bt = np.full((3, 4), -7, np.int32)
    bt[0, :2] = [5, 9]
    bt[2, :1] = [3]
    ctx, start, slots, pos, seq, head, bt2, bad = su.ref_plan(
        [20, 0, 16], [13, 0, 1], bt, np.array([7, 8, 1, 2]), 1, 16, 16, 16)
    assert ctx.tolist() == [33, 0, 17] and start.tolist() == [0, 13, 13, 14]
    assert bt2[0].tolist() == [5, 9, 8, -7] and bt2[2].tolist() == [3, 1, -7, -7]
    assert head == 3 and bad == 0
    assert slots.tolist() == [9 * 16 + o for o in range(4, 16)] + [8 * 16] + [16] + [-1, -1]
    assert pos.tolist() == list(range(20, 33)) + [16, 0, 0]
    assert seq.tolist() == [0] * 13 + [2, -1, -1]


def test_ref_table_by_hand():
    c, s = su.ref_table(0, 3, 4)
    assert np.allclose(c[:, 0], np.cos([0, 1, 2])) and np.allclose(s[:, 1], np.sin([0, .01, .02]))
    c2, _ = su.ref_table(0, 3, 4, scaling="linear", factor=2.0)
    assert np.allclose(c2[2], c[1])
    # yarn: the fastest column keeps its frequency, the slowest is interpolated
    w0, w1 = su.ref_freqs(128), su.ref_freqs(128, scaling="yarn", factor=8.0, orig_len=4096)
    assert w1[0] == w0[0] and np.isclose(float(w1[-1]), float(w0[-1]) / 8)
    # ntk: the slowest column is interpolated by exactly the factor
    w2 = su.ref_freqs(128, scaling="ntk", factor=4.0)
    assert np.isclose(float(w2[-1]), float(w0[-1]) / 4) and w2[0] == 1


def test_ref_turned_by_hand():
    x = np.array([[[3.0, 4.0, 1.0, 2.0]]])
    c, s = np.array([[0.0, 1.0]]), np.array([[1.0, 0.0]])  # a quarter turn, none
    y, _ = su.ref_turned(x, None, 0.0, c, s, 4, True)
    assert y.tolist() == [[[-4.0, 3.0, 1.0, 2.0]]]
    y, _ = su.ref_turned(x, None, 0.0, c, s, 4, False)
    assert y.tolist() == [[[-1.0, 4.0, 3.0, 2.0]]]
    y, _ = su.ref_turned(x, np.ones(4), 0.0, c[:, :0], s[:, :0], 0, True)
    assert np.allclose((y ** 2).mean(), 1.0)


def test_ref_attention_by_hand():
    k = np.zeros((2, 1, 16, 2))
    v = np.zeros((2, 1, 16, 2))
    k[1, 0, 0], k[1, 0, 1] = [1, 0], [0, 1]
    v[1, 0, 0], v[1, 0, 1] = [2, 0], [0, 4]
    q = np.array([[[np.log(3.0), 0.0]], [[0.0, 0.0]]])
    bt = np.array([[1], [1]])
    out, lse, *_ = su.ref_attention(q, k, v, bt, [2, 0], 1, 1.0)
    assert np.allclose(out[0, 0], [1.5, 1.0]) and np.isclose(lse[0, 0], np.log(4.0))
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all()
    out, lse, *_ = su.ref_attention(q, k, v, bt, [2, 0], 1, 1.0, topk=[[1, 1], [0, -1]])
    assert np.allclose(out[0, 0], [0.0, 4.0]) and np.isclose(lse[0, 0], np.log(2.0))
    out, _, *_ = su.ref_attention(q, k, v, bt, [2, 2], 1, 1.0, window=1)
    assert np.allclose(out[0, 0], [0.0, 4.0])
