"""The paged-cache operators against their 64-bit forms: attention of chunks and
single tokens over the pages, accumulated key weights, and eviction, at the
lengths, groups, page sizes, layouts and masks where they can go wrong.
Tolerances are derived in paged_reference."""

import math
import os
import subprocess
import sys
import threading

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
    attn.set_wait_timeout_ns(2_000_000_000)
    return attn_lib


def queries(lens, hq, d, dtype, seed, tail=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(sum(lens) + tail, hq, d, generator=g).to(dtype).cuda()


def ok():
    torch.cuda.synchronize()
    assert attn.get_error() == attn.ATTN_OK, hex(attn.last_device_error())


CHUNKS = [
    # new tokens, keys, Hq, Hkv, d, page, dtype, layout, causal
    ([1], [1], 1, 1, 64, 16, BF, "nhd", True),
    ([3, 0, 7], [5, 9, 7], 4, 2, 64, 16, BF, "nhd", True),
    ([130, 1, 64, 5], [130, 700, 65, 0], 8, 2, 128, 16, BF, "nhd", True),       # no keys at all
    ([200, 37], [150, 20], 4, 4, 128, 32, HF, "hnd", True),                     # rows that see no key
    ([257, 128, 127], [1000, 128, 300], 6, 2, 128, 64, HF, "joint", True),      # group 3
    ([33, 500], [2049, 513], 5, 1, 64, 128, BF, "nhd", True),                   # group 5
    ([90, 1, 256], [400, 256, 511], 8, 1, 128, 256, BF, "hnd", False),          # not causal, pages of two tiles
    ([40], [300], 71, 1, 64, 32, HF, "nhd", True),                              # a group of 71
    ([17, 3], [129, 1000], 160, 1, 64, 16, BF, "nhd", True),                    # a group wider than a tile
    ([4], [20000], 8, 2, 128, 16, BF, "nhd", True),                             # few rows over a long cache
    ([16, 1], [9000, 12345], 4, 1, 64, 64, HF, "joint", True),
    ([1024], [3000], 8, 2, 128, 32, BF, "nhd", True),
    ([1] * 70, [1 + 11 * i for i in range(70)], 4, 2, 64, 16, BF, "nhd", True),
    ([600, 0, 2, 900], [600, 77, 4000, 1500], 12, 12, 64, 16, HF, "nhd", False),
    # many blocks of queries, so that ranges start deep inside a chunk: fewer and more keys than queries
    ([3000, 700], [3001, 5000], 16, 1, 64, 64, BF, "nhd", True),
    ([2500, 1200], [900, 1300], 11, 1, 64, 32, HF, "nhd", True),
    ([1500], [4000], 32, 1, 128, 128, BF, "nhd", False),
    # more sequences than a block has threads
    ([i % 4 for i in range(700)], [(7 * i) % 90 for i in range(700)], 4, 2, 64, 16, HF, "nhd", True),
]


@pytest.mark.parametrize("case", CHUNKS, ids=[f"chunk{i}" for i in range(len(CHUNKS))])
def test_chunk(case):
    lq, lk, hq, hkv, d, page, dtype, layout, causal = case
    c = Cache(lk, hkv, d, page, dtype, seed=len(lq) + hq, layout=layout)
    q = queries(lq, hq, d, dtype, 5)
    scale = 1.0 / math.sqrt(d)
    o, lse = attn.attn_fwd_paged(q, *c.args(), cu_of(lq), causal=causal)
    ok()
    ref.check_attention(o, lse, q, c, lq, causal, scale)


def test_chunk_equals_the_packed_forward():
    lq, lk = [300, 17, 1], [900, 17, 400]
    c = Cache(lk, 2, 128, 32, BF, seed=3)
    q = queries(lq, 8, 128, BF, 4)
    o, lse = attn.attn_fwd_paged(q, *c.args(), cu_of(lq))
    k = torch.cat([c.rows(c.k, b) for b in range(3)])
    v = torch.cat([c.rows(c.v, b) for b in range(3)])
    pad = torch.zeros(128, 2, 128, dtype=BF, device="cuda")
    o2, lse2 = attn.attn_fwd(q, torch.cat((k, pad)), torch.cat((v, pad)), causal=True, cu_seqlens=cu_of(lq),
                             cu_seqlens_k=cu_of(lk))
    ok()
    assert float((o.float() - o2.float()).abs().max()) <= 2e-2
    assert float((lse - lse2).abs().max()) <= 1e-4


def test_chunk_leaves_other_rows_and_reads_no_other_rows():
    lq, lk = [5, 60], [200, 333]
    c = Cache(lk, 2, 64, 16, BF, seed=8)
    q = queries(lq, 4, 64, BF, 9, tail=40)
    q[65:] = float("nan")
    out = torch.full_like(q, 7.0)
    lse = torch.full((4, 105), 3.0, device="cuda")
    attn.attn_fwd_paged(q, *c.args(), cu_of(lq), out=out, lse=lse)
    ok()
    ref.check_attention(out[:65], lse[:, :65], q[:65], c, lq, True, 0.125)
    assert bool((out[65:] == 7.0).all()) and bool((lse[:, 65:] == 3.0).all())


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan"), -65504.0])
def test_chunk_masked_keys_of_any_value(value):
    # the chunk's last tokens are hidden from its first ones: their keys and
    # values may hold anything
    c = Cache([140], 1, 64, 16, HF, seed=2)
    q = queries([20], 2, 64, HF, 3)
    o, lse = attn.attn_fwd_paged(q, *c.args(), cu_of([20]))
    j = torch.arange(139, 140, device="cuda")
    page, slot = c.table[0, j // 16].long(), j % 16
    c.v[page, slot] = value
    o2, lse2 = attn.attn_fwd_paged(q, *c.args(), cu_of([20]))
    c.k[page, slot] = value
    o3, lse3 = attn.attn_fwd_paged(q, *c.args(), cu_of([20]))
    ok()
    if math.isfinite(value):
        assert torch.equal(o[:19], o2[:19])
    assert torch.equal(lse[:, :19], lse2[:, :19]) and torch.equal(lse[:, :19], lse3[:, :19])


DECODES = [
    # keys, Hq, Hkv, d, page, dtype, layout
    ([1], 1, 1, 64, 16, BF, "nhd"),
    ([0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257], 4, 2, 64, 16, BF, "nhd"),
    ([0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257], 4, 2, 128, 16, HF, "hnd"),
    ([4097, 3000, 1], 32, 8, 128, 16, BF, "nhd"),
    ([5000, 12], 6, 2, 128, 32, HF, "joint"),               # group 3
    ([700, 3], 5, 1, 64, 64, BF, "nhd"),
    ([1000, 260], 16, 1, 128, 128, BF, "hnd"),              # group 16
    ([513, 2], 24, 1, 64, 256, HF, "nhd"),                  # a group of 24: two parts
    ([129], 71, 1, 128, 16, BF, "nhd"),
    ([70000], 8, 2, 128, 64, BF, "nhd"),                    # cut over every SM
    ([70000], 4, 4, 64, 16, HF, "nhd"),
    ([33 * i % 611 for i in range(500)], 4, 2, 64, 16, BF, "nhd"),
    ([20000] + [3] * 40, 8, 1, 128, 32, BF, "nhd"),         # one long among many short
    ([0, 0, 0], 2, 1, 64, 16, BF, "nhd"),
    # key/value heads side by side in groups: 32 in four of 8, 14 at once, a prime number, none that fits
    ([3000, 17, 900], 32, 32, 64, 16, HF, "nhd"),
    ([2000, 1], 28, 14, 128, 32, BF, "nhd"),
    ([5000, 300], 7, 7, 64, 64, HF, "hnd"),
    ([1200, 640], 74, 37, 64, 16, BF, "nhd"),
    ([(5 * i) % 41 for i in range(5000)], 2, 1, 64, 16, HF, "nhd"),
]


@pytest.mark.parametrize("case", DECODES, ids=[f"decode{i}" for i in range(len(DECODES))])
def test_decode(case):
    lk, hq, hkv, d, page, dtype, layout = case
    c = Cache(lk, hkv, d, page, dtype, seed=len(lk) + hq, layout=layout)
    q = queries([1] * len(lk), hq, d, dtype, 6)
    o, lse = attn.attn_decode_paged(q, *c.args())
    ok()
    ref.check_attention(o, lse, q, c, [1] * len(lk), True, 1.0 / math.sqrt(d))


def test_decode_values_of_any_magnitude():
    for v_scale in (1e5, 1e-6):
        c = Cache([40000, 700], 2, 128, 32, BF, seed=3, v_scale=v_scale)
        q = queries([1, 1], 8, 128, BF, 6)
        o, lse = attn.attn_decode_paged(q, *c.args())
        ok()
        ref.check_attention(o, lse, q, c, [1, 1], True, 1.0 / math.sqrt(128))


@pytest.mark.parametrize("decode", [False, True])
def test_growing_scores_and_scale(decode):
    # scores that grow along the keys by far more than the softmax may defer a
    # rescaling, and scale 0 (every key the same weight)
    for scale, gain in ((2.0, 1.0), (0.0, 1.0)):
        c = Cache([900], 1, 64, 16, BF, seed=5)
        j = torch.arange(900, device="cuda")
        c.k[c.table[0, j // 16].long(), j % 16] *= (gain * (1 + j / 300.0))[:, None, None].to(BF)
        lens = [1] if decode else [300]
        q = queries(lens, 2, 64, BF, 6)
        if decode:
            o, lse = attn.attn_decode_paged(q, *c.args(), scale=scale)
        else:
            o, lse = attn.attn_fwd_paged(q, *c.args(), cu_of(lens), scale=scale)
        ok()
        ref.check_attention(o, lse, q, c, lens, True, scale)


def test_table_slices_shared_pages_and_wide_strides():
    # a slice of a wider table, two sequences on the same pages, and pages far
    # apart: offsets past 2^31 elements
    d, page, hkv = 128, 64, 2
    n = 40
    wide = torch.empty((n, 70_000_000), dtype=BF, device="cuda")   # 2.8e9 elements
    k = wide[:, : page * hkv * d].unflatten(1, (page, hkv, d))
    v = wide[:, page * hkv * d: 2 * page * hkv * d].unflatten(1, (page, hkv, d))
    g = torch.Generator().manual_seed(1)
    k.copy_(torch.randn(n, page, hkv, d, generator=g))
    v.copy_(torch.randn(n, page, hkv, d, generator=g))
    table = torch.full((2, 50), -1, dtype=torch.int32, device="cuda")
    table[0, 10:50] = torch.arange(39, -1, -1, device="cuda")
    table[1, 10:50] = torch.arange(39, -1, -1, device="cuda")
    c = Cache([1], hkv, d, page, BF, seed=1)
    c.lens, c.k, c.v, c.table = [2500, 900], k, v, table[:, 10:]
    c.seqlens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    q = queries([1, 1], 8, d, BF, 6)
    o, lse = attn.attn_decode_paged(q, *c.args())
    ok()
    ref.check_attention(o, lse, q, c, [1, 1], True, 1.0 / math.sqrt(d))
    q = queries([20, 3], 8, d, BF, 6)
    o, lse = attn.attn_fwd_paged(q, *c.args(), cu_of([20, 3]))
    ok()
    ref.check_attention(o, lse, q, c, [20, 3], True, 1.0 / math.sqrt(d))
    w = attn.key_weights(q, k, lse, c.table, c.seqlens, cu_of([20, 3]))
    ok()
    check_weights(w, None, q, c, lse, [20, 3], True, 1.0 / math.sqrt(d), 0.0)


def check_weights(w, before, q, c, lse, lq, causal, scale, decay):
    """Bar: the score's error and that of exp's argument (fp32: |scaled score -
    lse| 2^-22), the exponential and the sum of up to m G terms; and what was
    there, scaled and rounded."""
    at = 0
    for b, m in enumerate(lq):
        n = c.lens[b]
        k = c.rows(c.k, b)
        r = ref.key_weights(q[at:at + m], k, lse[:, at:at + m], causal, scale)
        old = before[b, :, :n].double() * decay if before is not None else torch.zeros_like(r)
        rel = 2 * ref.score_error(q[at:at + m], k, scale) + 2.0 ** -16 + m * (q.shape[1] // c.hkv) * 2.0 ** -24
        bar = rel * r + (r + old.abs()) * 2.0 ** -22 + 1e-30
        err = (w[b, :, :n].double() - (r + old)).abs()
        assert bool((err <= bar).all()), (b, float((err / bar).max()))
        at += m


WEIGHTS = [
    # new tokens, keys, Hq, Hkv, d, page, dtype, layout, causal, decay
    ([1], [1], 1, 1, 64, 16, BF, "nhd", True, 1.0),
    ([1, 1, 1], [0, 129, 4000], 8, 2, 128, 16, BF, "nhd", True, 1.0),
    ([1] * 40, [37 * i for i in range(40)], 4, 2, 64, 16, HF, "hnd", True, 0.5),
    ([130, 0, 5], [400, 200, 5], 6, 2, 64, 32, HF, "joint", True, 0.0),
    ([300, 40], [150, 40], 5, 1, 128, 64, BF, "nhd", True, 0.9),       # rows that see no key
    ([700], [2000], 8, 2, 128, 128, BF, "nhd", True, 1.0),
    ([100, 333], [777, 1025], 12, 12, 64, 256, BF, "hnd", False, 1.0),
    ([20], [500], 71, 1, 64, 32, HF, "nhd", True, 1.0),
    ([9, 3], [300, 70], 160, 1, 64, 16, BF, "nhd", True, 0.0),
    ([2, 900, 1], [3000, 900, 64], 4, 1, 128, 16, BF, "nhd", True, 1.0),
    # ranges that start deep inside a long cache, few and many queries a tile
    ([900, 3], [12000, 9000], 4, 2, 64, 128, HF, "nhd", True, 1.0),
    ([1500], [9500], 3, 1, 64, 64, HF, "nhd", False, 0.5),
    ([2000], [700], 20, 1, 64, 32, HF, "nhd", True, 1.0),
    ([i % 3 for i in range(900)], [(7 * i) % 90 for i in range(900)], 4, 2, 64, 16, HF, "nhd", True, 1.0),
    ([1, 2], [3000, 700], 24, 1, 64, 16, BF, "nhd", True, 1.0),
    ([1] * 3, [2000, 17, 900], 64, 32, 64, 16, HF, "nhd", True, 1.0),
    ([40, 1], [2000, 300], 7, 7, 128, 64, BF, "hnd", True, 0.0),
]


@pytest.mark.parametrize("case", WEIGHTS, ids=[f"weights{i}" for i in range(len(WEIGHTS))])
def test_key_weights(case):
    lq, lk, hq, hkv, d, page, dtype, layout, causal, decay = case
    c = Cache(lk, hkv, d, page, dtype, seed=len(lq) + hq, layout=layout)
    q = queries(lq, hq, d, dtype, 7, tail=9)
    q[sum(lq):] = float("nan")
    scale = 1.0 / math.sqrt(d)
    lse = torch.full((hq, q.shape[0]), float("nan"), device="cuda")
    attn.attn_fwd_paged(q, *c.args(), cu_of(lq), causal=causal, lse=lse)
    w = torch.rand(len(lq), hkv, c.table.shape[1] * page, device="cuda")
    if decay == 0.0:
        w[:] = float("nan")   # what was there is not read
    before = w.clone()
    got = attn.key_weights(q, c.k, lse, c.table, c.seqlens, cu_of(lq), causal=causal, decay=decay, weights=w)
    ok()
    assert got is w
    for b, n in enumerate(lk):
        assert torch.equal(w[b, :, n:].nan_to_num(-1.0), before[b, :, n:].nan_to_num(-1.0))
    check_weights(w, None if decay == 0.0 else before, q, c, lse, lq, causal, scale, decay)
    # the weights of each query sum to one over the keys, of each head
    if decay == 0.0 and causal:
        for b, (m, n) in enumerate(zip(lq, lk)):
            total = float(w[b, :, :n].double().sum())
            seen = min(m, n) * hq
            assert abs(total - seen) <= 1e-4 * max(seen, 1)


def test_key_weights_default_buffer_and_decode_form():
    lk = [100, 0, 1000]
    c = Cache(lk, 2, 128, 32, BF, seed=4)
    q = queries([1, 1, 1], 8, 128, BF, 2)
    o, lse = attn.attn_decode_paged(q, *c.args())
    w = attn.key_weights(q, c.k, lse, c.table, c.seqlens, cu_of([1, 1, 1]))
    w2 = attn.key_weights(q, c.k, lse, c.table, c.seqlens, cu_of([1, 1, 1]), weights=w.clone())
    ok()
    check_weights(w, None, q, c, lse, [1, 1, 1], True, 1.0 / math.sqrt(128), 0.0)
    assert bool((w[0, :, 100:] == 0).all()) and bool((w[1] == 0).all())
    assert torch.allclose(w2, 2 * w, rtol=2.0 ** -22)


EVICTS = [
    # keys, Hkv, d, page, dtype, budget, recent, layout
    ([1], 1, 64, 16, BF, 1, 0, "nhd"),
    ([10, 0, 3, 11], 2, 64, 16, BF, 4, 1, "nhd"),
    ([300, 100, 299, 5000], 2, 128, 16, HF, 100, 0, "hnd"),
    ([300, 100, 299, 5000], 3, 128, 32, BF, 100, 100, "joint"),      # only the recent keys
    ([2000, 2001, 1999], 1, 64, 64, BF, 2000, 37, "nhd"),
    ([70000], 2, 128, 128, BF, 5001, 1000, "nhd"),
    ([4096] * 5, 4, 128, 256, HF, 2048, 256, "nhd"),
    ([33 * i % 611 for i in range(90)], 2, 64, 16, BF, 64, 7, "nhd"),
]


def evict_weights(c, n, kind, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(len(c.lens), c.hkv, n, generator=g) ** 4
    if kind == "ties":
        w = (w * 4).floor() / 4
    elif kind == "same":
        w = torch.full_like(w, 0.25)
    elif kind == "odd":   # negative, infinite, NaN, both zeros, tiny
        pick = torch.randint(0, 8, w.shape, generator=g)
        for i, x in enumerate((float("inf"), -float("inf"), float("nan"), -0.0, 0.0, 1e-42, -1.5)):
            w[pick == i] = x
    return w.cuda()


@pytest.mark.parametrize("kind", ["plain", "ties", "same", "odd"])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("case", EVICTS, ids=[f"evict{i}" for i in range(len(EVICTS))])
def test_evict(case, in_place, kind):
    lk, hkv, d, page, dtype, budget, recent, layout = case
    c = Cache(lk, hkv, d, page, dtype, seed=len(lk), layout=layout, poison=False,
              spare=2 + sum(-(-min(n, budget) // page) for n in lk))
    w = evict_weights(c, c.table.shape[1] * page, kind, 3)
    k0, v0 = c.k.clone(), c.v.clone()
    dst = None
    if not in_place:
        # the pool's pages that the table does not name; the first sequence keeps its first page in place
        used = set()
        for b, n in enumerate(lk):
            used |= set(c.table[b, : -(-n // page)].tolist())
        free = [x for x in range(c.n_pages) if x not in used]
        dst = torch.full((len(lk), max(1, -(-budget // page))), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(lk):
            m = -(-min(n, budget) // page)
            dst[b, :m] = torch.tensor(free[at:at + m], dtype=torch.int32)
            at += m
        if lk[0] > 0:
            dst[0, 0] = int(c.table[0, 0])
        dst = dst.cuda()
    kept, seqlens, wout = attn.cache_evict(w.clone(), c.k, c.v, c.table, c.seqlens, budget, recent, dst_page_table=dst)
    ok()
    assert seqlens.tolist() == [min(n, budget) for n in lk]
    where = c.table if dst is None else dst
    written = torch.zeros(c.n_pages, page, dtype=torch.bool, device="cuda")
    rows_w, rows_k = w.cpu(), kept.cpu()
    for b, n in enumerate(lk):
        m = min(n, budget)
        j = torch.arange(m, device="cuda")
        pg, sl = where[b, j // page].long(), j % page
        written[pg, sl] = True
        src = [c.table[b, : max(1, -(-n // page))].long()]
        for g in range(hkv):
            want = ref.evict(rows_w[b, g].tolist(), n, budget, recent)
            assert rows_k[b, g, :m].tolist() == want and rows_k[b, g, m:].tolist() == [-1] * (budget - m)
            idx = torch.tensor(want, dtype=torch.long, device="cuda")
            for new, old in ((c.k, k0), (c.v, v0)):
                assert torch.equal(new[pg, sl, g], old[src[0][idx // page], idx % page, g]) if m else True
            assert torch.equal(wout[b, g, :m].nan_to_num(5.0), w[b, g, idx].nan_to_num(5.0))
            assert bool((wout[b, g, m:] == 0).all())
    # nothing else in the pool has changed
    assert torch.equal(c.k[~written], k0[~written]) and torch.equal(c.v[~written], v0[~written])


@pytest.mark.parametrize("kind", ["plain", "ties"])
def test_evict_from_more_keys_than_a_cluster_holds(kind):
    n = 500_000
    c = Cache([n], 1, 64, 256, BF, seed=3, poison=False)
    w = evict_weights(c, c.table.shape[1] * 256, kind, 5)
    k0 = c.k.clone()
    kept, seqlens, wout = attn.cache_evict(w, c.k, c.v, c.table, c.seqlens, 7001, 1001)
    ok()
    want = ref.evict(w[0, 0].tolist(), n, 7001, 1001)
    assert seqlens.tolist() == [7001] and kept[0, 0].tolist() == want
    idx = torch.tensor(want, device="cuda")
    j = torch.arange(7001, device="cuda")
    got = c.k[c.table[0, j // 256].long(), j % 256]
    assert torch.equal(got, k0[c.table[0, idx // 256].long(), idx % 256])
    assert torch.equal(wout[0, 0], w[0, 0, idx])


def test_evict_weights_in_place():
    c = Cache([500, 80], 2, 64, 16, BF, seed=1, poison=False)
    w = evict_weights(c, 520, "plain", 1)
    w0 = w.clone()
    kept, seqlens, got = attn.cache_evict(w, c.k, c.v, c.table, c.seqlens, 100, 10, weights_out=w)
    ok()
    assert got is w
    for b, n in enumerate(c.lens):
        m = min(n, 100)
        for g in range(2):
            assert torch.equal(w[b, g, :m], w0[b, g, kept[b, g, :m].long()]) and bool((w[b, g, m:] == 0).all())


def test_a_serving_loop():
    """Prompt in chunks, weights, eviction, then decoding steps with the rotary
    positions running on: against the same loop in 64 bits on the rows the
    cache held."""
    B, hq, hkv, d, page, dtype = 3, 8, 2, 128, 16, BF
    prompt, chunk, budget, recent = [150, 61, 300], 128, 64, 16
    freqs, amp = attn.rotary_freqs(d, scaling="yarn", factor=4.0, original_len=128)
    width = 24
    n_pages = B * width
    k = torch.full((n_pages, page, hkv, d), float("nan"), dtype=dtype, device="cuda")
    v = k.clone()
    g = torch.Generator().manual_seed(2)
    table = torch.randperm(n_pages, generator=g).to(torch.int32).view(B, width).cuda()
    c = Cache([1] * B, hkv, d, page, dtype, seed=1)
    c.k, c.v, c.table = k, v, table
    weights = torch.zeros(B, hkv, width * page, device="cuda")
    lens, seen = [0] * B, [0] * B
    scale = 1.0 / math.sqrt(d)

    def step(new):
        cu, total = cu_of(new), sum(new)
        qkv = torch.randn(total, hq + 2 * hkv, d, generator=g).to(dtype).cuda()
        qr, kr, vr = qkv.split((hq, hkv, hkv), dim=1)
        for b in range(B):
            lens[b] += new[b]
        seqlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        pos = torch.cat([torch.arange(s, s + n) for s, n in zip(seen, new)]).to(torch.int32).cuda()
        q = attn.cache_append(kr, vr, k, v, table, seqlens, cu, q=qr, freqs=freqs, amplitude=amp, positions=pos)
        for b in range(B):
            seen[b] += new[b]
        c.lens, c.seqlens = list(lens), seqlens
        at = 0
        for b, n in enumerate(new):   # the tokens are where they belong, turned
            ref.check_turn(c.rows(k, b)[lens[b] - n:], kr[at:at + n], pos[at:at + n], freqs, amp, False)
            assert torch.equal(c.rows(v, b)[lens[b] - n:], vr[at:at + n])
            at += n
        ref.check_turn(q, qr, pos, freqs, amp, False)
        if max(new) == 1 and min(new) == 1:
            o, lse = attn.attn_decode_paged(q, k, v, table, seqlens)
        else:
            o, lse = attn.attn_fwd_paged(q, k, v, table, seqlens, cu)
        ok()
        ref.check_attention(o, lse, q, c, new, True, scale)
        before = weights.clone()
        attn.key_weights(q, k, lse, table, seqlens, cu, decay=0.9, weights=weights)
        ok()
        check_weights(weights, before, q, c, lse, new, True, scale, 0.9)
        return seqlens

    left = list(prompt)
    while any(left):
        new = [min(chunk, x) for x in left]
        left = [x - n for x, n in zip(left, new)]
        seqlens = step(new)
    for _ in range(2):
        before = weights.clone()
        kept, seqlens, _ = attn.cache_evict(weights, k, v, table, seqlens, budget, recent, weights_out=weights)
        ok()
        for b in range(B):
            for h in range(hkv):
                want = ref.evict(before[b, h].tolist(), lens[b], budget, recent)
                assert kept[b, h, :len(want)].tolist() == want
            lens[b] = min(lens[b], budget)
        for _ in range(3):
            seqlens = step([1] * B)


def test_two_streams_and_two_graphs():
    """The same shapes on two streams at once, and two captured graphs replayed
    at once: no scratch memory is shared."""
    cases = []
    for seed in (1, 2):
        c = Cache([30000, 500], 2, 128, 16, BF, seed=seed)
        q1 = queries([1, 1], 8, 128, BF, seed)
        q2 = queries([40, 300], 8, 128, BF, seed + 5)
        cases.append((c, q1, q2, cu_of([40, 300])))

    def both(c, q1, q2, cu, stream=None):
        o1, l1 = attn.attn_decode_paged(q1, *c.args(), stream=stream)
        o2, l2 = attn.attn_fwd_paged(q2, *c.args(), cu, stream=stream)
        w = attn.key_weights(q2, c.k, l2, c.table, c.seqlens, cu, stream=stream)
        kept, n, _ = attn.cache_evict(w, c.k, c.v, c.table, c.seqlens, 1 << 20, stream=stream)   # (moves nothing)
        return o1, l1, o2, l2, w, kept[..., :100].clone(), n

    want = [both(*x) for x in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = [both(*x, stream=s) for x, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    graphs, outs = [], []
    for x in cases:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(both(*x))
        graphs.append(gr)
    for _ in range(5):
        for out in outs:
            for t in out:
                t.fill_(1.0)
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    ok()


def test_two_threads_on_one_stream():
    """Calls of two threads that interleave on a stream: each has its own
    scratch memory between its kernels."""
    cs = [Cache([40000, 500], 2, 128, 16, BF, seed=s) for s in (1, 2)]
    qs = [queries([1, 1], 8, 128, BF, s) for s in (1, 2)]
    want = [attn.attn_decode_paged(q, *c.args()) for c, q in zip(cs, qs)]
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        got[i] = [attn.attn_decode_paged(qs[i], *cs[i].args()) for _ in range(200)]

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1]) for o, lse in got[i])
    ok()


def test_many_streams_and_eager_calls_beside_a_graph():
    c = Cache([20000, 500], 2, 64, 16, BF, seed=1)
    q = queries([1, 1], 8, 64, BF, 1)
    want = attn.attn_decode_paged(q, *c.args())
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = attn.attn_decode_paged(q, *c.args())
    streams = [torch.cuda.Stream() for _ in range(12)]   # more than the kept scratch buffers
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        gr.replay()
        for s in streams:
            got.append(attn.attn_decode_paged(q, *c.args(), stream=s))
        torch.cuda.synchronize()
        for o, lse in got + [out]:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    ok()


def test_the_first_call_of_a_process_is_captured():
    # nothing of the library has run before the capture
    script = """
import torch
from tests.paged_reference import Cache, check_attention, cu_of
from tiled_attention_attn_gb300 import attn
c = Cache([3000, 70], 2, 64, 32, torch.float16, seed=1)
q = torch.randn(42, 4, 64, generator=torch.Generator().manual_seed(1)).half().cuda()
cu = cu_of([40, 2])
f, a = attn.rotary_freqs(64)
torch.cuda.synchronize()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    r = attn.cache_append(q[:, :2], q[:, 2:], *c.args(), cu, q=q, freqs=f, amplitude=a)
    o, lse = attn.attn_fwd_paged(r, *c.args(), cu)
    o2, lse2 = attn.attn_decode_paged(r[:2], *c.args())
    w = attn.key_weights(r, c.k, lse, c.table, c.seqlens, cu)
for _ in range(2):
    gr.replay()
torch.cuda.synchronize()
assert attn.get_error() == 0
check_attention(o, lse, r, c, [40, 2], True, 0.125)
check_attention(o2, lse2, r[:2], c, [1, 1], True, 0.125)
assert abs(float(w.double().sum()) - 42 * 4) < 1e-2
print("done")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", script], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stdout + r.stderr


def test_the_same_inputs_give_the_same_bits():
    c = Cache([9000, 77, 4000], 2, 128, 16, BF, seed=3)
    q1, q2, cu = queries([1] * 3, 8, 128, BF, 3), queries([100, 5, 700], 8, 128, BF, 4), cu_of([100, 5, 700])
    first = None
    for _ in range(4):
        o1, l1 = attn.attn_decode_paged(q1, *c.args())
        o2, l2 = attn.attn_fwd_paged(q2, *c.args(), cu)
        w = attn.key_weights(q2, c.k, l2, c.table, c.seqlens, cu)
        got = (o1, l1, o2, l2, w)
        first = got if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    ok()


def expect_error(code):
    assert attn.get_error() == attn.ATTN_EDEVICE
    assert attn.last_device_error() == code
    assert attn.get_error() == attn.ATTN_OK


@pytest.mark.parametrize("bad", [-1, 1 << 29])
def test_bad_lengths_are_reported(bad):
    c = Cache([100, 200], 1, 64, 16, BF, seed=1)
    q = queries([1, 1], 2, 64, BF, 1)
    c.seqlens[0] = bad
    o, lse = attn.attn_decode_paged(q, *c.args())
    expect_error(attn.ATTN_DEVERR_BAD_SEQLENS)
    assert bool((o[0] == 0).all()) and bool((lse[:, 0] == -float("inf")).all())
    good = Cache([0, 200], 1, 64, 16, BF, seed=1)
    good.k, good.v, good.table = c.k, c.v, c.table
    ref.check_attention(o, lse, q, good, [1, 1], True, 0.125)
    o, lse = attn.attn_fwd_paged(q, *c.args(), cu_of([1, 1]))
    expect_error(attn.ATTN_DEVERR_BAD_SEQLENS)
    ref.check_attention(o, lse, q, good, [1, 1], True, 0.125)
    w = torch.full((2, 1, c.table.shape[1] * 16), 2.0, device="cuda")
    attn.key_weights(q, c.k, lse, c.table, c.seqlens, cu_of([1, 1]), weights=w)
    expect_error(attn.ATTN_DEVERR_BAD_SEQLENS)
    assert bool((w[0] == 2.0).all())
    kept, seqlens, _ = attn.cache_evict(w, c.k, c.v, c.table, c.seqlens, 50)
    expect_error(attn.ATTN_DEVERR_BAD_SEQLENS)
    assert seqlens.tolist() == [0, 50]


def test_bad_offsets_are_reported():
    c = Cache([100, 200], 1, 64, 16, BF, seed=1)
    q = queries([6], 2, 64, BF, 1)
    for cu in ([0, 4, 3], [0, 4, 9], [-2, 3, 6]):
        t = torch.tensor(cu, dtype=torch.int32, device="cuda")
        attn.attn_fwd_paged(q, *c.args(), t)
        expect_error(attn.ATTN_DEVERR_BAD_SEQLENS)
        attn.key_weights(q, c.k, torch.zeros(2, 6, device="cuda"), c.table, c.seqlens, t)
        expect_error(attn.ATTN_DEVERR_BAD_SEQLENS)


@pytest.mark.parametrize("bad", [-1, 1 << 20, -(1 << 31)])
def test_bad_pages_are_reported(bad):
    c = Cache([100, 200], 1, 64, 16, BF, seed=1)
    q = queries([1, 1], 2, 64, BF, 1)
    c.table[0, 2] = bad
    good = ref.attention(q[1:], c.rows(c.k, 1), c.rows(c.v, 1), True, 0.125)[0]
    for f in (lambda: attn.attn_decode_paged(q, *c.args()), lambda: attn.attn_fwd_paged(q, *c.args(), cu_of([1, 1]))):
        o, lse = f()
        expect_error(attn.ATTN_DEVERR_BAD_PAGE)
        assert float((o[1].double() - good[0]).abs().max()) <= 2e-2
    attn.key_weights(q, c.k, lse, c.table, c.seqlens, cu_of([1, 1]))
    expect_error(attn.ATTN_DEVERR_BAD_PAGE)
    w = torch.zeros(2, 1, c.table.shape[1] * 16, device="cuda")
    attn.cache_evict(w, c.k, c.v, c.table, c.seqlens, 60, 30)
    expect_error(attn.ATTN_DEVERR_BAD_PAGE)
