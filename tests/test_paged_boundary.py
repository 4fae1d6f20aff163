"""Refusals of the paged-cache entry points, before anything reaches a GPU, and
the scaled rotary spectra."""

import ctypes
import math

import pytest
import torch

from tiled_attention_attn_gb300 import attn
from tiled_attention_attn_gb300.paged import _PagedKV

F = ctypes.c_float
GOOD = dict(k=256, v=256, page_table=16, seqlens_k=16, stride_page=4096, stride_token=128, stride_head=64,
            table_stride=4, max_pages=4, num_pages=10, page_size=16, num_kv_heads=2, head_dim=64, fp16=0)
CACHE_BAD = [dict(k=None), dict(v=None), dict(page_table=None), dict(seqlens_k=None), dict(k=264), dict(v=8),
             dict(stride_page=0), dict(stride_token=-128), dict(stride_head=60), dict(stride_page=1 << 40),
             dict(table_stride=3), dict(max_pages=0), dict(num_pages=0), dict(num_kv_heads=0), dict(fp16=2),
             dict(max_pages=1 << 27, table_stride=1 << 27)]
CACHE_UNSUPPORTED = [dict(head_dim=96), dict(head_dim=256), dict(page_size=8), dict(page_size=48), dict(page_size=512)]


def cache(**kw):
    return ctypes.byref(_PagedKV(**{**GOOD, **kw}))


def fwd(L, c=None, q=16, o=16, lse=16, B=2, Hq=4, total=8, cu=16, causal=1, scale=0.125, ws=256, n=1 << 40):
    return L.attn_fwd_paged(q, o, lse, B, Hq, total, c or cache(), cu, causal, F(scale), ws, n, None)


def decode(L, c=None, q=16, o=16, lse=16, B=2, Hq=4, scale=0.125, ws=256, n=1 << 40):
    return L.attn_decode_paged(q, o, lse, B, Hq, c or cache(), F(scale), ws, n, None)


def weights(L, c=None, q=16, lse=16, w=16, n=64, B=2, Hq=4, total=8, cu=16, causal=1, scale=0.125, decay=1.0, ws=256,
            m=1 << 40):
    return L.attn_key_weights(q, lse, w, n, B, Hq, total, c or cache(), cu, causal, F(scale), F(decay), ws, m, None)


def evict(L, c=None, w=16, n=64, kept=16, lens=32, wo=48, no=64, B=2, dst=None, ds=0, dm=0, budget=8, recent=2):
    return L.attn_cache_evict(w, n, kept, lens, wo, no, B, c or cache(), dst, ds, dm, budget, recent, None)


FREQS = (ctypes.c_double * 32)(*[0.5] * 32)


def append(L, c=None, q=4096, k=16, v=16, q_out=16, sq=256, sk=128, sv=128, B=2, Hq=4, total=2, cu=16, rot=64,
           f=FREQS, amp=1.0, inter=0, pos=None):
    return L.attn_cache_append(q, k, v, q_out, sq, sk, sv, B, Hq, total, c or cache(), cu, rot, f, F(amp), inter, pos,
                               None)


def rope(L, x=16, y=1 << 20, B=1, Ln=4, H=2, d=64, rot=64, f=FREQS, amp=1.0, inter=0, inv=0, st=128, sh=64, cu=None,
         total=0, off=None, pos=None, fp16=0):
    return L.attn_rotary_scaled(x, y, B, Ln, H, d, rot, f, F(amp), inter, inv, st, sh, cu, total, off, pos, fp16, None)


@pytest.mark.parametrize("call", [fwd, decode, append, evict, weights])
@pytest.mark.parametrize("bad", CACHE_BAD, ids=str)
def test_bad_caches(attn_lib, call, bad):
    if call is weights and "v" in bad:
        pytest.skip("the weights do not read the values")
    assert call(attn_lib, c=cache(**bad)) == attn.ATTN_EINVAL


@pytest.mark.parametrize("call", [fwd, decode, append, evict, weights])
@pytest.mark.parametrize("bad", CACHE_UNSUPPORTED, ids=str)
def test_unsupported_caches(attn_lib, call, bad):
    assert call(attn_lib, c=cache(**bad)) == attn.ATTN_EUNSUPPORTED


@pytest.mark.parametrize("call", [fwd, decode, append, evict, weights])
@pytest.mark.parametrize("B", [0, -1, 65536])
def test_bad_batch(attn_lib, call, B):
    assert call(attn_lib, B=B) == attn.ATTN_EINVAL


COMMON = [dict(q=None), dict(q=8), dict(lse=None), dict(lse=2), dict(Hq=0), dict(Hq=3), dict(scale=-1.0),
          dict(scale=math.nan), dict(scale=math.inf)]


@pytest.mark.parametrize("bad", COMMON + [dict(o=None), dict(o=24), dict(cu=None), dict(total=-1), dict(causal=2),
                                          dict(total=1 << 30, Hq=1 << 10), dict(ws=None), dict(ws=128), dict(n=0)],
                         ids=str)
def test_chunk_refusals(attn_lib, bad):
    assert fwd(attn_lib, **bad) == attn.ATTN_EINVAL


@pytest.mark.parametrize("bad", COMMON + [dict(o=None), dict(o=24), dict(ws=None), dict(ws=128), dict(n=0)], ids=str)
def test_decode_refusals(attn_lib, bad):
    assert decode(attn_lib, **bad) == attn.ATTN_EINVAL


@pytest.mark.parametrize("bad", COMMON + [dict(w=None), dict(w=2), dict(n=0), dict(cu=None), dict(total=-1),
                                          dict(causal=-1), dict(decay=math.nan), dict(decay=math.inf),
                                          dict(ws=None), dict(ws=128), dict(m=0)], ids=str)
def test_weights_refusals(attn_lib, bad):
    assert weights(attn_lib, **bad) == attn.ATTN_EINVAL


@pytest.mark.parametrize("bad", [dict(w=None), dict(kept=None), dict(lens=None), dict(wo=None), dict(w=2), dict(n=0),
                                 dict(no=7), dict(budget=0), dict(recent=9), dict(recent=-1), dict(lens=16),
                                 dict(wo=16, no=32), dict(dst=16, ds=1, dm=2), dict(dst=16, ds=4, dm=0),
                                 dict(dst=16, ds=1, dm=1, budget=17, no=17)], ids=str)
def test_evict_refusals(attn_lib, bad):
    assert evict(attn_lib, **bad) == attn.ATTN_EINVAL


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(q=None), dict(q_out=None), dict(q=4104), dict(k=24),
                                 dict(sq=255), dict(sk=120), dict(sv=129), dict(Hq=0), dict(cu=None), dict(total=-1),
                                 dict(rot=0), dict(rot=63), dict(rot=66), dict(f=None), dict(amp=math.nan),
                                 dict(inter=2), dict(q_out=4096 + 512), dict(q=4096, q_out=4096, sq=512)], ids=str)
def test_append_refusals(attn_lib, bad):
    assert append(attn_lib, **bad) == attn.ATTN_EINVAL


@pytest.mark.parametrize("bad", [dict(x=None), dict(y=None), dict(B=0), dict(Ln=-1), dict(H=0), dict(d=0), dict(rot=0),
                                 dict(rot=7), dict(rot=66), dict(f=None), dict(amp=math.inf), dict(inter=2),
                                 dict(inv=2), dict(st=63), dict(sh=63), dict(fp16=2), dict(pos=16, off=16),
                                 dict(pos=16, cu=16), dict(y=16 + 64), dict(x=16, y=16, st=256), dict(x=17),
                                 dict(cu=16, total=-1), dict(B=1 << 16, Ln=1 << 16)], ids=str)
def test_rotary_refusals(attn_lib, bad):
    assert rope(attn_lib, **bad) == attn.ATTN_EINVAL


def test_frequencies_must_be_finite(attn_lib):
    for x in (math.nan, math.inf):
        assert rope(attn_lib, f=(ctypes.c_double * 32)(*[0.1] * 31 + [x])) == attn.ATTN_EINVAL


def test_nothing_to_do(attn_lib):
    assert fwd(attn_lib, total=0) == attn.ATTN_OK
    assert append(attn_lib, total=0) == attn.ATTN_OK
    assert rope(attn_lib, Ln=0) == attn.ATTN_OK


def test_workspace_query_refusals(attn_lib):
    assert attn_lib.attn_paged_workspace_bytes(96, 0) == attn.ATTN_EUNSUPPORTED
    assert attn_lib.attn_paged_workspace_bytes(64, 3) == attn.ATTN_EINVAL


def test_binding_refuses_host_tensors_and_wrong_types():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 1], dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_fwd_paged(q, k, k, table, lens, cu)
    with pytest.raises(TypeError):
        attn.attn_decode_paged(q, k.float(), k.float(), table, lens)
    with pytest.raises(ValueError):
        attn.cache_append(q[:, :2], q[:, :2], k, k, table, lens, cu)
    with pytest.raises(ValueError):
        attn.key_weights(q, k, torch.zeros(4, 1), table, lens, cu)
    with pytest.raises(ValueError):
        attn.cache_evict(torch.zeros(1, 2, 64), k, k, table, lens, 8)
    f, a = attn.rotary_freqs(64)
    with pytest.raises(TypeError):
        attn.rotary_scaled(q.float(), f, a)
    with pytest.raises(ValueError):
        attn.rotary_scaled(q, f, a, positions=lens)


def test_scaled_spectra():
    plain, one = attn.rotary_freqs(128)
    assert one == 1.0 and plain[0] == 1.0 and abs(float(plain[-1]) - 10000.0 ** (-126 / 128)) < 1e-18
    lin, one = attn.rotary_freqs(128, scaling="linear", factor=4.0)
    assert one == 1.0 and torch.allclose(lin * 4.0, plain, rtol=1e-15)
    ntk, one = attn.rotary_freqs(128, scaling="ntk", factor=4.0)
    assert one == 1.0 and float(ntk[0]) == 1.0 and abs(float(ntk[-1] * 4.0 / plain[-1]) - 1.0) < 1e-12
    yarn, amp = attn.rotary_freqs(128, scaling="yarn", factor=4.0, original_len=4096)
    assert abs(amp - (0.1 * math.log(4.0) + 1.0)) < 1e-15
    turns = plain * 4096 / (2 * math.pi)
    assert torch.equal(yarn[turns > 40], plain[turns > 40])
    assert torch.allclose(yarn[turns < 0.8] * 4.0, plain[turns < 0.8], rtol=1e-12)
    between = (yarn <= plain) & (yarn >= plain / 4.0 * (1 - 1e-12))
    assert bool(between.all())
    assert attn.rotary_freqs(2, scaling="ntk", factor=4.0)[0].tolist() == [1.0]
    for kw in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=64, base=1.0), dict(rot_dim=64, factor=0.5),
               dict(rot_dim=64, scaling="other")):
        with pytest.raises(ValueError):
            attn.rotary_freqs(**kw)
