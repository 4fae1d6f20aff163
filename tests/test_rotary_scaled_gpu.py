"""Rotary embedding with scaled frequencies, its gradient, and the append of new
tokens to a paged cache, against 64-bit forms (tolerances in paged_reference)."""

import math

import pytest
import torch

from . import paged_reference as ref
from .paged_reference import Cache, cu_of
from tiled_attention_attn_gb300 import attn

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib(attn_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return attn_lib


def rand(*shape, dtype, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


CASES = [
    # leading shape, H, d, rot, interleaved, dtype, scaling
    ((1,), 1, 64, 64, False, BF, "yarn"),
    ((37,), 3, 128, 128, True, HF, "ntk"),
    ((2, 300), 5, 128, 64, False, HF, "linear"),
    ((3, 77), 4, 128, 112, True, BF, None),
    ((1, 33), 2, 64, 30, True, BF, "yarn"),        # pairs past whole 16-byte words
    ((2, 19), 3, 50, 50, False, HF, "ntk"),        # rows past whole 16-byte words
    ((5000,), 1, 64, 48, False, BF, "linear"),
    ((2, 2000), 32, 128, 128, False, BF, "yarn"),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[f"case{i}" for i in range(len(CASES))])
def test_rotation_at_far_positions(case, inverse):
    lead, H, d, rot, inter, dtype, scaling = case
    x = rand(*lead, H, d, dtype=dtype)
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(-100, 1 << 20, lead, generator=g, dtype=torch.int32)
    pos.view(-1)[0] = (1 << 31) - 1
    f, a = attn.rotary_freqs(rot, scaling=scaling, factor=8.0, original_len=2048)
    y = attn.rotary_scaled(x, f, a, interleaved=inter, positions=pos.cuda(), inverse=inverse)
    torch.cuda.synchronize()
    # positions up to 2^31: the 64-bit reference's own product is exact to 2^-22 there
    ref.check_turn(y.view(-1, H, d), x.view(-1, H, d), pos.view(-1).cuda(), f, a, inter, -1.0 if inverse else 1.0)
    z = x.clone()
    assert attn.rotary_scaled(z, f, a, interleaved=inter, positions=pos.cuda(), inverse=inverse, out=z) is z
    torch.cuda.synchronize()
    assert torch.equal(z, y)


def test_offsets_packed_rows_and_strides():
    f, a = attn.rotary_freqs(64, scaling="linear", factor=4.0)
    lens = [5, 0, 40, 1]
    x = rand(60, 3, 64, dtype=BF)
    off = torch.tensor([7, 3, 100000, 0], dtype=torch.int32).cuda()
    out = torch.full_like(x, 9.0)
    attn.rotary_scaled(x, f, a, cu_seqlens=cu_of(lens), offsets=off, out=out)
    torch.cuda.synchronize()
    pos = torch.cat([torch.arange(n) + int(o) for n, o in zip(lens, off)]).cuda()
    ref.check_turn(out[:46], x[:46], pos, f, a, False)
    assert bool((out[46:] == 9.0).all())
    # dense, offsets per sequence, the middle part of a fused projection
    qkv = rand(2, 50, 12, 64, dtype=HF)
    part = qkv[:, :, 4:8]
    y = attn.rotary_scaled(part, f, a, offsets=torch.tensor([0, 900], dtype=torch.int32).cuda())
    swapped = qkv.transpose(1, 2).contiguous().transpose(1, 2)     # heads before tokens
    with pytest.raises(ValueError):
        attn.rotary_scaled(swapped, f, a)                          # batch and length not evenly strided
    y1 = attn.rotary_scaled(swapped[:1], f, a)
    torch.cuda.synchronize()
    pos = torch.cat((torch.arange(50), torch.arange(50) + 900)).cuda()
    ref.check_turn(y.view(100, 4, 64), part.reshape(100, 4, 64), pos, f, a, False)
    ref.check_turn(y1.view(50, 12, 64), swapped[0], pos[:50], f, a, False)


def test_equals_the_unscaled_rotary():
    x = rand(2, 100, 4, 128, dtype=BF)
    f, a = attn.rotary_freqs(128)
    y, z = attn.rotary_scaled(x, f, a), attn.rotary(x)
    torch.cuda.synchronize()
    assert float((y.float() - z.float()).abs().max()) <= 2.0 ** -5


@pytest.mark.parametrize("inter", [False, True])
def test_gradient(inter):
    f, a = attn.rotary_freqs(48, scaling="yarn", factor=4.0, original_len=512)
    x = rand(2, 30, 3, 64, dtype=HF).requires_grad_()
    off = torch.tensor([50, 7000], dtype=torch.int32).cuda()
    dy = rand(2, 30, 3, 64, dtype=HF, seed=4)
    y = attn.rotary_scaled_func(x, f, a, inter, offsets=off)
    y.backward(dy)
    pos = torch.cat((torch.arange(30) + 50, torch.arange(30) + 7000)).cuda()
    # the formula: the transposed rotation
    ref.check_turn(x.grad.view(60, 3, 64), dy.view(60, 3, 64), pos, f, a, inter, -1.0)
    # and differences of the 64-bit forward along a direction (it is linear, so any step serves)
    e = rand(60, 3, 64, dtype=HF, seed=5)
    xx = x.detach().view(60, 3, 64).double()
    step = ref.turn(xx + e.double(), pos, f, a, inter) - ref.turn(xx, pos, f, a, inter)
    want = float((step * dy.view(60, 3, 64).double()).sum())
    got = float((x.grad.view(60, 3, 64).double() * e.double()).sum())
    bar = float((x.grad.double().abs().view(60, 3, 64) * e.double().abs()).sum()) * 2.0 ** -10 + 1e-6
    assert abs(got - want) <= bar


def test_gradient_of_an_expanded_output_and_of_packed_rows():
    f, a = attn.rotary_freqs(64)
    x = rand(20, 2, 64, dtype=BF).requires_grad_()
    y = attn.rotary_scaled_func(x, f, a, cu_seqlens=cu_of([5, 9]))
    y.sum().backward()     # the gradient arrives as an expanded scalar
    torch.cuda.synchronize()
    assert bool((y[14:] == 0).all()) and bool((x.grad[14:] == 0).all())
    one = torch.ones(14, 2, 64, dtype=BF, device="cuda")
    pos = torch.cat((torch.arange(5), torch.arange(9))).cuda()
    ref.check_turn(x.grad[:14], one, pos, f, a, False, -1.0)


def test_gradient_of_the_gradient():
    # the operator is linear: d/dx of <R^T dy, e> with respect to dy is R e
    f, a = attn.rotary_freqs(64, scaling="ntk", factor=4.0)
    x = rand(1, 21, 2, 64, dtype=HF).requires_grad_()
    dy = rand(1, 21, 2, 64, dtype=HF, seed=3).requires_grad_()
    e = rand(1, 21, 2, 64, dtype=HF, seed=4)
    g, = torch.autograd.grad(attn.rotary_scaled_func(x, f, a), x, dy, create_graph=True)
    gg, = torch.autograd.grad(g, dy, e)
    torch.cuda.synchronize()
    ref.check_turn(gg.view(21, 2, 64), e.view(21, 2, 64), torch.arange(21).cuda(), f, a, False)


def test_backward_in_a_graph_beside_an_eager_one():
    f, a = attn.rotary_freqs(64, scaling="linear", factor=2.0)
    x = rand(1, 40, 2, 64, dtype=BF).requires_grad_()
    dy = rand(1, 40, 2, 64, dtype=BF, seed=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            want, = torch.autograd.grad(attn.rotary_scaled_func(x, f, a), x, dy)
    torch.cuda.current_stream().wait_stream(s)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got, = torch.autograd.grad(attn.rotary_scaled_func(x, f, a), x, dy)
    got.fill_(0)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


APPENDS = [
    # new tokens, keys after them, Hq, Hkv, d, rot, page, dtype, layout, interleaved
    ([1], [1], 2, 1, 64, 64, 16, BF, "nhd", False),
    ([1, 1, 0, 1], [17, 4000, 9, 16], 8, 2, 128, 128, 16, BF, "nhd", False),
    ([300, 5, 64], [300, 40, 1000], 6, 3, 128, 64, 32, HF, "hnd", True),
    ([33, 0, 129], [500, 0, 129], 4, 4, 64, 64, 64, HF, "joint", False),
    ([900], [2000], 32, 8, 128, 112, 256, BF, "nhd", True),
    ([7, 20], [50, 30], 3, 1, 64, 30, 128, BF, "nhd", True),     # pairs past whole 16-byte words
]


@pytest.mark.parametrize("case", APPENDS, ids=[f"append{i}" for i in range(len(APPENDS))])
@pytest.mark.parametrize("turned", [True, False])
def test_append(case, turned):
    lq, lk, hq, hkv, d, rot, page, dtype, layout, inter = case
    c = Cache(lk, hkv, d, page, dtype, seed=1, layout=layout)
    k0, v0 = c.k.clone(), c.v.clone()
    total = sum(lq)
    qkv = rand(total + 3, hq + 2 * hkv, d, dtype=dtype, seed=2)
    q, k, v = qkv.split((hq, hkv, hkv), dim=1)
    key = torch.cat([torch.arange(n - m, n) for m, n in zip(lq, lk)]).cuda()
    f, a = attn.rotary_freqs(rot, scaling="yarn", factor=4.0, original_len=256)
    q_out = torch.full((total + 3, hq, d), 5.0, dtype=dtype, device="cuda")
    pos = key
    if turned:
        pos = torch.cat((key + 1000, torch.zeros(3, dtype=torch.long, device="cuda"))).to(torch.int32)
        got = attn.cache_append(k, v, *c.args(), cu_of(lq), q=q, freqs=f, amplitude=a, interleaved=inter,
                                positions=pos, q_out=q_out)
        assert got is q_out
    else:
        assert attn.cache_append(k, v, *c.args(), cu_of(lq)) is None
    torch.cuda.synchronize()
    assert attn.get_error() == attn.ATTN_OK
    written = torch.zeros(c.n_pages, page, dtype=torch.bool, device="cuda")
    at = 0
    for b, (m, n) in enumerate(zip(lq, lk)):
        j = torch.arange(n - m, n, device="cuda")
        pg, sl = c.table[b, j // page].long(), j % page
        written[pg, sl] = True
        assert torch.equal(c.v[pg, sl], v[at:at + m])
        if turned:
            ref.check_turn(c.k[pg, sl], k[at:at + m], pos[at:at + m], f, a, inter)
        else:
            assert torch.equal(c.k[pg, sl], k[at:at + m])
        at += m
    if turned:
        ref.check_turn(q_out[:total], q[:total], pos[:total], f, a, inter)
        assert bool((q_out[total:] == 5.0).all())
    for new, old in ((c.k, k0), (c.v, v0)):
        assert torch.equal(new[~written].nan_to_num(77.0), old[~written].nan_to_num(77.0))


def test_append_rotates_q_in_place_at_the_key_index():
    c = Cache([40, 9], 2, 64, 16, BF, seed=1)
    q, k, v = rand(12, 4, 64, dtype=BF, seed=3), rand(12, 2, 64, dtype=BF, seed=4), rand(12, 2, 64, dtype=BF, seed=5)
    q0 = q.clone()
    f, a = attn.rotary_freqs(32)
    attn.cache_append(k, v, *c.args(), cu_of([8, 4]), q=q, freqs=f, amplitude=a, q_out=q)
    torch.cuda.synchronize()
    key = torch.cat((torch.arange(32, 40), torch.arange(5, 9))).cuda()
    ref.check_turn(q, q0, key, f, a, False)
    ref.check_turn(c.rows(c.k, 1)[5:], k[8:], key[8:], f, a, False)


def test_append_reports_bad_places():
    def expect(code):
        assert attn.get_error() == attn.ATTN_EDEVICE and attn.last_device_error() == code
    f, a = attn.rotary_freqs(64)
    k, v = rand(6, 1, 64, dtype=BF), rand(6, 1, 64, dtype=BF, seed=1)
    c = Cache([100, 3], 1, 64, 16, BF, seed=1)
    k0 = c.k.clone()
    attn.cache_append(k, v, *c.args(), cu_of([2, 4]))              # 4 new tokens of 3 keys
    expect(attn.ATTN_DEVERR_BAD_SEQLENS)
    c.k.copy_(k0)
    c.table[0, 6] = c.n_pages
    attn.cache_append(k, v, *c.args(), cu_of([6, 0]))              # tokens 96 .. 99 on no page
    expect(attn.ATTN_DEVERR_BAD_PAGE)
    changed = (c.k.nan_to_num(7.0) != k0.nan_to_num(7.0)).flatten(1).any(1)
    assert int(changed.sum()) == 1                                 # tokens 94 and 95 alone
    for cu in ([0, 5, 3], [0, 2, 7]):
        attn.cache_append(k, v, *c.args(), torch.tensor(cu, dtype=torch.int32).cuda())
        assert attn.get_error() == attn.ATTN_EDEVICE
    c.seqlens[0] = 1 << 30
    attn.cache_append(k, v, *c.args(), cu_of([6, 0]))
    expect(attn.ATTN_DEVERR_BAD_SEQLENS)
