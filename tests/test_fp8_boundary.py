"""Refusals of the entry points of head norms and of caches of 8-bit floating
point, before anything reaches a GPU."""

import ctypes
import math

import pytest
import torch

from tiled_attention_attn_gb300 import attn
from tiled_attention_attn_gb300.fp8 import _PagedKV8

F = ctypes.c_float
GOOD = dict(k=256, v=256, k_scales=16, v_scales=16, page_table=16, seqlens_k=16, stride_page=4096, stride_token=128,
            stride_head=64, scale_stride_page=32, scale_stride_token=2, scale_stride_head=1, table_stride=4, max_pages=4,
            num_pages=10, page_size=16, num_kv_heads=2, head_dim=64)
CACHE_BAD = [dict(k=None), dict(v=None), dict(k_scales=None), dict(v_scales=None), dict(page_table=None),
             dict(seqlens_k=None), dict(k=264), dict(v=8), dict(k_scales=6), dict(stride_page=0), dict(stride_token=-128),
             dict(stride_head=72), dict(stride_page=1 << 40), dict(scale_stride_page=0), dict(scale_stride_token=-1),
             dict(scale_stride_head=1 << 40), dict(table_stride=3), dict(max_pages=0), dict(num_pages=0),
             dict(num_kv_heads=0), dict(max_pages=1 << 27, table_stride=1 << 27)]
CACHE_UNSUPPORTED = [dict(head_dim=96), dict(head_dim=256), dict(page_size=8), dict(page_size=48), dict(page_size=512)]
FREQS = (ctypes.c_double * 32)(*[0.5] * 32)


def cache(**kw):
    return ctypes.byref(_PagedKV8(**{**GOOD, **kw}))


def append(L, c=None, q=4096, k=16, v=16, q_out=16, sq=256, sk=128, sv=128, B=2, Hq=4, total=2, cu=16, rot=64, f=FREQS,
           amp=1.0, inter=0, pos=None, fp16=0):
    return L.attn_cache_append_fp8(q, k, v, q_out, sq, sk, sv, B, Hq, total, c or cache(), cu, rot, f, F(amp), inter, pos,
                                   fp16, None)


def read(L, c=None, k=16, v=1 << 20, B=2, total=8, cu=16, starts=None, fp16=0):
    return L.attn_cache_read_fp8(k, v, B, total, c or cache(), cu, starts, fp16, None)


def tree(L, c=None, q=16, o=1 << 20, lse=16, B=2, Hq=4, total=8, most=8, cu=16, mask=None, scale=0.125, fp16=0, ws=256,
         n=1 << 40):
    return L.attn_tree_fp8(q, o, lse, B, Hq, total, most, c or cache(), cu, mask, F(scale), fp16, ws, n, None)


@pytest.mark.parametrize("call", [append, read, tree])
@pytest.mark.parametrize("bad", CACHE_BAD, ids=str)
def test_bad_caches(attn_lib, call, bad):
    assert call(attn_lib, c=cache(**bad)) == attn.ATTN_EINVAL


@pytest.mark.parametrize("call", [append, read, tree])
@pytest.mark.parametrize("bad", CACHE_UNSUPPORTED, ids=str)
def test_unsupported_caches(attn_lib, call, bad):
    assert call(attn_lib, c=cache(**bad)) == attn.ATTN_EUNSUPPORTED


@pytest.mark.parametrize("call", [append, read, tree])
@pytest.mark.parametrize("B", [0, -1, 65536])
def test_bad_batch(attn_lib, call, B):
    assert call(attn_lib, B=B) == attn.ATTN_EINVAL


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(q=None), dict(q_out=None), dict(q=4104), dict(k=24),
                                 dict(sq=255), dict(sk=120), dict(sv=129), dict(Hq=0), dict(cu=None), dict(total=-1),
                                 dict(rot=0), dict(rot=63), dict(rot=66), dict(f=None), dict(amp=math.nan), dict(inter=2),
                                 dict(fp16=2), dict(q_out=4096 + 512), dict(q=4096, q_out=4096, sq=512),
                                 dict(f=(ctypes.c_double * 32)(*[0.1] * 31 + [math.inf]))], ids=str)
def test_append_refusals(attn_lib, bad):
    assert append(attn_lib, **bad) == attn.ATTN_EINVAL


def test_append_of_other_rotary_dimensions(attn_lib):
    assert append(attn_lib, rot=40) == attn.ATTN_EUNSUPPORTED


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(k=24), dict(cu=None), dict(total=-1), dict(fp16=2),
                                 dict(v=16 + 1024)], ids=str)
def test_read_refusals(attn_lib, bad):
    assert read(attn_lib, **bad) == attn.ATTN_EINVAL


@pytest.mark.parametrize("bad", [dict(q=None), dict(q=8), dict(o=None), dict(o=24), dict(lse=None), dict(lse=2), dict(Hq=0),
                                 dict(Hq=3), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(most=0),
                                 dict(most=65), dict(cu=None), dict(total=-1), dict(mask=12), dict(fp16=3),
                                 dict(total=1 << 30, Hq=1 << 10), dict(ws=None), dict(ws=128), dict(n=0),
                                 dict(o=16), dict(o=16 + 64)], ids=str)
def test_tree_refusals(attn_lib, bad):
    assert tree(attn_lib, **bad) == attn.ATTN_EINVAL


def norm(L, q=16, k=1 << 16, qo=1 << 20, ko=1 << 24, sq=256, hq=64, sk=128, hk=64, rows=4, Hq=4, Hk=2, d=64, wq=None,
         wk=None, w32=0, eps=1e-6, rot=64, f=FREQS, axis=None, axes=1, amp=1.0, inter=0, pos=16, fp16=0):
    return L.attn_qk_norm_rotary(q, k, qo, ko, sq, hq, sk, hk, rows, Hq, Hk, d, wq, wk, w32, F(eps), rot, f, axis, axes,
                                 F(amp), inter, pos, fp16, None)


def norm_bwd(L, dqo=1 << 26, dko=1 << 27, q=16, k=1 << 16, qo=1 << 20, ko=1 << 24, dwq=16, dwk=16, sq=256, hq=64, sk=128,
             hk=64, rows=4, Hq=4, Hk=2, d=64, wq=16, wk=16, w32=0, eps=1e-6, rot=64, f=FREQS, axis=None, axes=1, amp=1.0,
             inter=0, pos=16, fp16=0, ws=256, n=1 << 40):
    return L.attn_qk_norm_rotary_bwd(dqo, dko, q, k, qo, ko, dwq, dwk, sq, hq, sk, hk, rows, Hq, Hk, d, wq, wk, w32, F(eps),
                                     rot, f, axis, axes, F(amp), inter, pos, fp16, ws, n, None)


def ints(*x):
    return (ctypes.c_int * len(x))(*x)


NORM_BAD = [dict(q=None), dict(k=None), dict(q=8), dict(k=(1 << 16) + 2), dict(qo=None), dict(ko=None), dict(qo=24),
            dict(sq=63), dict(sq=260), dict(hq=60), dict(hq=68), dict(sk=1 << 41), dict(rows=-1), dict(Hq=0), dict(Hk=-1),
            dict(d=0), dict(d=-64), dict(wq=8), dict(wk=24), dict(w32=2), dict(eps=-1.0), dict(eps=math.nan), dict(rot=-16),
            dict(rot=63), dict(rot=80), dict(f=None), dict(axes=0), dict(axes=9), dict(axis=ints(*[0] * 31, 1)),
            dict(axis=ints(*[-1] * 32), axes=2), dict(amp=math.inf), dict(inter=2), dict(pos=None), dict(pos=18),
            dict(fp16=2), dict(qo=16 + 64), dict(ko=16), dict(qo=1 << 24), dict(q=16, qo=16, sq=512),
            dict(f=(ctypes.c_double * 32)(*[math.nan] * 32))]


@pytest.mark.parametrize("call", [norm, norm_bwd])
@pytest.mark.parametrize("bad", NORM_BAD, ids=str)
def test_norm_refusals(attn_lib, call, bad):
    assert call(attn_lib, **bad) == attn.ATTN_EINVAL


@pytest.mark.parametrize("call", [norm, norm_bwd])
@pytest.mark.parametrize("other", [dict(d=72, hq=72, hk=72, sq=288, sk=144), dict(rot=40),
                                   dict(d=528, hq=528, hk=528, sq=4 * 528, sk=2 * 528)], ids=str)
def test_unsupported_norms(attn_lib, call, other):
    assert call(attn_lib, **other) == attn.ATTN_EUNSUPPORTED


@pytest.mark.parametrize("bad", [dict(dqo=None), dict(dko=None), dict(dqo=(1 << 26) + 8), dict(dqo=(1 << 20) + 512),
                                 dict(dko=1 << 20), dict(dwq=17), dict(dwk=18, w32=1), dict(ws=None), dict(ws=128),
                                 dict(n=0)], ids=str)
def test_norm_backward_refusals(attn_lib, bad):
    assert norm_bwd(attn_lib, **bad) == attn.ATTN_EINVAL


def test_nothing_to_do(attn_lib):
    assert append(attn_lib, total=0) == attn.ATTN_OK
    assert read(attn_lib, total=0) == attn.ATTN_OK
    assert tree(attn_lib, total=0) == attn.ATTN_OK
    assert norm(attn_lib, rows=0) == attn.ATTN_OK


def test_workspace_query_refusals(attn_lib):
    assert attn_lib.attn_fp8_workspace_bytes(96) == attn.ATTN_EUNSUPPORTED
    assert attn_lib.attn_qk_norm_workspace_bytes(0) == attn.ATTN_EINVAL
    assert attn_lib.attn_qk_norm_workspace_bytes(72) == attn.ATTN_EUNSUPPORTED


def test_binding_refuses_host_tensors_and_wrong_types():
    k8 = torch.zeros(4, 16, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros(4, 16, 2)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 1], dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_decode_fp8(q, k8, k8, s, s, table, lens)
    with pytest.raises(TypeError):
        attn.attn_decode_fp8(q, k8.view(torch.uint8), k8.view(torch.uint8), s, s, table, lens)
    with pytest.raises(ValueError):
        attn.attn_tree_fp8(q, k8, k8, s, s, table, lens, cu)
    with pytest.raises(ValueError):
        attn.attn_tree_fp8(q, k8, k8, s, s, table, lens, None)
    with pytest.raises(ValueError):
        attn.cache_read_fp8(k8, k8, s, s, table, lens, cu, 1)
    with pytest.raises(ValueError):
        attn.cache_append_fp8(q[:, :2], q[:, :2], k8, k8, s, s, table, lens, cu)
    f, _ = attn.rotary_freqs(64)
    with pytest.raises(ValueError):
        attn.qk_norm_rotary(q)
    with pytest.raises(TypeError):
        attn.qk_norm_rotary(q.float())
    with pytest.raises(TypeError):
        attn.qk_norm_rotary_func(q, q.half(), None, None, f, lens)
