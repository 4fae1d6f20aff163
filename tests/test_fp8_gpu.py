"""The operators over caches of 8-bit floating point against their 64-bit forms:
append, reading back, and attention of single tokens and trees, at the lengths,
groups, page sizes, layouts and masks where they can go wrong.  Tolerances are
derived in fp8_reference."""

import math
import threading

import pytest
import torch

from . import fp8_reference as ref
from .fp8_reference import E4M3, Cache8, bits_of, cu_of, random_trees
from tiled_attention_attn_gb300 import attn

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib(attn_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.set_wait_timeout_ns(2_000_000_000)
    return attn_lib


def queries(n, hq, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, hq, d, generator=g).to(dtype).cuda()


def ok():
    torch.cuda.synchronize()
    assert attn.get_error() == attn.ATTN_OK, hex(attn.last_device_error())


# ------------------------------------------------------------------ append

APPENDS = [
    # new tokens, keys, Hq, Hkv, d, page, dtype, layout, rot, interleaved
    ([1], [1], 1, 1, 64, 16, BF, "nhd", 64, False),
    ([1, 1, 1], [5, 700, 33], 8, 2, 128, 16, BF, "nhd", 128, False),
    ([3, 0, 70], [5, 9, 70], 4, 2, 64, 32, HF, "hnd", 32, True),
    ([130, 17], [1000, 17], 6, 3, 128, 64, HF, "joint", 64, False),
    ([33, 500, 1], [2049, 513, 256], 5, 5, 128, 256, BF, "hnd", 112, True),
    ([700, 1300], [900, 1300], 32, 8, 64, 128, BF, "nhd", 64, True),
    ([2000], [2000], 71, 1, 64, 16, HF, "nhd", 16, False),
    ([i % 3 for i in range(300)], [i % 3 + i for i in range(300)], 2, 1, 128, 16, BF, "nhd", 128, False),
]


def check_rows(pages, scales, at, x, slack):
    """Quantised rows at `at` against x (64-bit): the scale within `slack` of the row,
    each value within half an e4m3 step and that."""
    top = x.abs().amax(-1)
    s = scales[at].double()
    assert bool(((s - (top / 448.0).clamp(min=2.0 ** -126)).abs() <= (slack.amax(-1) + top * 2.0 ** -23) / 448.0).all())
    got = pages.view(torch.uint8)[at].view(E4M3).double() * s[..., None]
    y = x / s[..., None]
    bar = s[..., None] * ref.half_step8(y * (1 + 2.0 ** -18)) * (1 + 2.0 ** -20) + slack + x.abs() * 2.0 ** -22
    err = (got - x).abs()
    assert bool((err <= bar).all()), float((err / bar).max())


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("case", APPENDS, ids=[f"append{i}" for i in range(len(APPENDS))])
def test_append(case, fused):
    lq, lk, hq, hkv, d, page, dtype, layout, rot, inter = case
    c = Cache8(lk, hkv, d, page, seed=len(lq) + hq, layout=layout)
    total = sum(lq)
    qkv = queries(total, hq + 2 * hkv, d, dtype, 5) * 3
    q, k, v = qkv.split((hq, hkv, hkv), dim=1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    freqs, amp = attn.rotary_freqs(rot, scaling="yarn", factor=8.0)
    before = c.snapshot()
    q_out = attn.cache_append_fp8(k, v, *c.args(), cu_of(lq), q=q, freqs=freqs, amplitude=amp, interleaved=inter)
    ok()
    kept = torch.ones(c.k.shape[:2], dtype=torch.bool, device="cuda")
    at = 0
    for b, m in enumerate(lq):
        n = lk[b]
        pos = torch.arange(n - m, n)
        place = c.places(b, m, n - m)
        kept[place] = False
        turned = ref.turn(k[at:at + m], pos, freqs, amp, inter)
        norm = ref.turn(k[at:at + m].abs().amax(-1, keepdim=True).expand(-1, -1, d), torch.zeros_like(pos), freqs, 1.0, inter)
        check_rows(c.k, c.ks, place, turned, 2.0 ** -19 * amp * norm)
        v8, vs = ref.quantise(v[at:at + m])
        assert torch.equal(c.v.view(torch.uint8)[place], v8.view(torch.uint8)) and torch.equal(c.vs[place], vs)
        at += m
    from .paged_reference import check_turn
    pos = torch.cat([torch.arange(n - m, n) for m, n in zip(lq, lk)])
    check_turn(q_out, q, pos, freqs, amp, inter)
    # no other slot changed
    for t, old in zip((c.k.view(torch.uint8), c.v.view(torch.uint8), c.ks, c.vs), before):
        assert torch.equal(t[kept].nan_to_num(7.0) if t.dtype == torch.float32 else t[kept],
                           old[kept].nan_to_num(7.0) if t.dtype == torch.float32 else old[kept])


def test_append_positions_and_no_rotation():
    lq, lk = [5, 40], [90, 41]
    c, plain = Cache8(lk, 2, 128, 16, 1), Cache8(lk, 2, 128, 16, 1)
    k, v, q = (queries(45, h, 128, BF, s) for h, s in ((2, 1), (2, 2), (4, 3)))
    freqs, amp = attn.rotary_freqs(128)
    pos = torch.randint(-100000, 1 << 31, (45,), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    out = attn.cache_append_fp8(k, v, *c.args(), cu_of(lq), q=q, freqs=freqs, positions=pos.cuda(), q_out=q.clone())
    assert attn.cache_append_fp8(k, v, *plain.args(), cu_of(lq)) is None
    ok()
    from .paged_reference import check_turn
    check_turn(out, q, pos, freqs, amp, False)
    at = 0
    for b, (m, n) in enumerate(zip(lq, lk)):
        place = c.places(b, m, n - m)
        turned = ref.turn(k[at:at + m], pos[at:at + m], freqs, amp, False)
        check_rows(c.k, c.ks, place, turned, 2.0 ** -19 * k[at:at + m].double().abs().amax(-1, keepdim=True).expand_as(turned))
        k8, ks = ref.quantise(k[at:at + m])
        assert torch.equal(plain.k.view(torch.uint8)[place], k8.view(torch.uint8)) and torch.equal(plain.ks[place], ks)
        at += m


@pytest.mark.parametrize("dtype", [BF, HF])
def test_append_of_extreme_rows(dtype):
    # zeros, subnormals, the largest values, powers of two (quotients on the border of two e4m3 values), NaN, infinities
    d, tiny = 64, torch.finfo(dtype).smallest_normal
    g = torch.Generator().manual_seed(1)
    rows = torch.zeros(16, d)
    rows[1, 3] = tiny
    rows[2] = torch.randn(d, generator=g) * tiny / 8
    rows[3] = torch.randn(d, generator=g).sign() * torch.finfo(dtype).max
    rows[4] = 2.0 ** -torch.arange(d).float()
    rows[5] = torch.arange(d).float() / 64
    rows[5, 0] = 1.0
    rows[6] = torch.arange(d).float() * 0.75
    rows[7, 5] = math.nan
    rows[8, 0] = math.inf
    rows[9, 63] = -math.inf
    rows[10] = 448.0
    rows[11] = torch.arange(d).float() - 30.5
    rows[12:] = torch.randn(4, d, generator=g) * torch.tensor([1e-4, 1.0, 30.0, 3e4])[:, None]
    x = rows.to(dtype).cuda()[:, None].expand(-1, 2, -1).contiguous()
    c = Cache8([16], 2, d, 16, 3)
    attn.cache_append_fp8(x, x, *c.args(), cu_of([16]))
    ok()
    place = c.places(0)
    v8, vs = ref.quantise(x)
    for pages, scales in ((c.k, c.ks), (c.v, c.vs)):
        assert torch.equal(pages.view(torch.uint8)[place] & 0x7f, v8.view(torch.uint8) & 0x7f)
        assert torch.equal(scales[place].isnan(), vs.isnan()) and torch.equal(scales[place].nan_to_num(), vs.nan_to_num())
    k, _ = attn.cache_read_fp8(*c.args(), cu_of([16]), 16, dtype)
    ok()
    bad = ~torch.isfinite(x).all(-1, keepdim=True).expand_as(x)   # (of the last row in fp16 too: 2.2 times 3e4 is infinite)
    assert bool(bad[7:10].all()) and torch.equal(k.isnan(), bad)


def test_append_of_more_tokens_than_keys_and_bad_offsets():
    c = Cache8([4, 30], 1, 64, 16, 1)
    before = c.snapshot()
    k = queries(20, 1, 64, BF, 1)
    attn.cache_append_fp8(k, k, *c.args(), cu_of([6, 3]))       # two of the six tokens have no key
    torch.cuda.synchronize()
    assert attn.get_error() == attn.ATTN_EDEVICE and attn.last_device_error() == attn.ATTN_DEVERR_BAD_SEQLENS
    k8, _ = ref.quantise(k)
    assert torch.equal(c.k.view(torch.uint8)[c.places(0)], k8.view(torch.uint8)[2:6])
    assert torch.equal(c.k.view(torch.uint8)[c.places(1, 3, 27)], k8.view(torch.uint8)[6:9])
    bad = Cache8([4, 30], 1, 64, 16, 1)
    attn.cache_append_fp8(k, k, *bad.args(), torch.tensor([0, 40, 3], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert attn.get_error() == attn.ATTN_EDEVICE
    assert torch.equal(bad.k.view(torch.uint8), before[0])


# ------------------------------------------------------------------ read

@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens, hkv, d, page, layout", [
    ([1], 1, 64, 16, "nhd"), ([5, 0, 700], 2, 128, 16, "hnd"), ([257, 33], 5, 64, 256, "joint"),
    ([3000, 1, 513], 8, 128, 64, "nhd"), ([i % 5 for i in range(400)], 1, 64, 16, "nhd"),
])
def test_read(lens, hkv, d, page, layout, dtype):
    c = Cache8(lens, hkv, d, page, 2, layout)
    total = sum(lens)
    marks = [torch.full((total + 3, hkv, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    k, v = attn.cache_read_fp8(*c.args(), cu_of(lens), total + 3, dtype, k_out=marks[0], v_out=marks[1])
    ok()
    for got, which in ((k, "k"), (v, "v")):
        want = torch.cat([x * s[..., None] for x, s in (c.rows(b, which) for b in range(len(lens)))]).to(dtype)
        assert torch.equal(got[:total], want)
        assert bool((got[total:] == 7.0).all())   # rows behind the last sequence


def test_read_of_parts():
    lens = [300, 41, 90]
    c = Cache8(lens, 2, 64, 32, 4)
    starts, counts = [299, 0, 17], [1, 40, 60]
    k, v = attn.cache_read_fp8(*c.args(), cu_of(counts), 101, HF, starts=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    ok()
    for got, which in ((k, "k"), (v, "v")):
        want = torch.cat([(x * s[..., None])[a:a + m] for (x, s), a, m in
                          zip((c.rows(b, which) for b in range(3)), starts, counts)]).to(HF)
        assert torch.equal(got, want)


def test_read_past_the_last_key():
    c = Cache8([10, 20], 1, 64, 16, 4)
    out = torch.full((24, 1, 64), 7.0, dtype=BF, device="cuda")
    starts = torch.tensor([2, -1], dtype=torch.int32, device="cuda")
    k, _ = attn.cache_read_fp8(*c.args(), cu_of([12, 12]), 24, BF, starts=starts, k_out=out)
    torch.cuda.synchronize()
    assert attn.get_error() == attn.ATTN_EDEVICE and attn.last_device_error() == attn.ATTN_DEVERR_BAD_SEQLENS
    x, s = c.rows(0, "k")
    assert torch.equal(k[:8], (x * s[..., None])[2:].to(BF)) and bool((k[8:13] == 7.0).all())
    x, s = c.rows(1, "k")
    assert torch.equal(k[13:], (x * s[..., None])[:11].to(BF))


# ------------------------------------------------------------------ attention

DECODES = [
    # keys, Hq, Hkv, d, page, dtype, layout
    ([1], 1, 1, 64, 16, BF, "nhd"),
    ([0, 1, 128, 129], 2, 2, 128, 16, HF, "nhd"),
    ([5, 300, 0, 2049], 8, 2, 64, 16, BF, "hnd"),
    ([5, 300, 0, 2049], 8, 2, 128, 32, BF, "joint"),
    ([255, 256, 257], 6, 2, 64, 64, HF, "nhd"),
    ([1000, 64], 5, 1, 128, 128, HF, "hnd"),
    ([4097], 8, 1, 128, 256, BF, "nhd"),
    ([20000], 32, 8, 128, 16, BF, "nhd"),
    ([33000, 5], 16, 4, 64, 64, HF, "nhd"),
    ([700], 71, 1, 64, 32, BF, "nhd"),              # a wide odd group
    ([300, 129], 160, 1, 128, 16, HF, "nhd"),       # wider than one tile
    ([1 + 11 * i for i in range(70)], 4, 2, 64, 16, BF, "nhd"),
    ([(7 * i) % 90 for i in range(700)], 4, 2, 128, 16, HF, "nhd"),
    ([513] * 3, 40, 5, 128, 16, BF, "nhd"),
]


@pytest.mark.parametrize("case", DECODES, ids=[f"decode{i}" for i in range(len(DECODES))])
def test_decode(case):
    lens, hq, hkv, d, page, dtype, layout = case
    c = Cache8(lens, hkv, d, page, seed=len(lens) + hq, layout=layout)
    q = queries(len(lens), hq, d, dtype, 6)
    o, lse = attn.attn_decode_fp8(q, *c.args())
    ok()
    ref.check_attention(o, lse, q, c, [1] * len(lens), None, 1.0 / math.sqrt(d))


TREES = [
    # tokens, keys, Hq, Hkv, d, page, dtype, layout, max_tokens
    ([1], [1], 1, 1, 64, 16, BF, "nhd", 1),
    ([2, 0, 5], [2, 9, 300], 4, 2, 128, 16, HF, "nhd", None),
    ([7, 3], [129, 130], 8, 2, 64, 32, BF, "hnd", 7),
    ([12, 1, 9], [140, 500, 256], 16, 4, 128, 64, BF, "joint", 16),
    ([64], [64], 2, 2, 64, 16, HF, "nhd", 64),
    ([64, 40], [700, 1100], 8, 2, 128, 16, BF, "nhd", None),
    ([64, 63, 1], [3000, 63, 200], 12, 2, 64, 128, HF, "nhd", 64),
    ([33], [5000], 32, 8, 128, 256, BF, "nhd", 33),
    ([5], [30000], 5, 1, 128, 16, HF, "hnd", 5),
    ([9, 4], [4, 100], 4, 1, 64, 16, BF, "nhd", 9),           # more tokens than keys
    ([2, 3, 0, 1] * 60, [(13 * i) % 200 + 4 for i in range(240)], 4, 2, 64, 16, BF, "nhd", 3),
    ([3, 17], [400, 900], 71, 1, 64, 32, HF, "nhd", 17),
    ([2], [131], 160, 1, 128, 16, BF, "nhd", 2),
]


@pytest.mark.parametrize("kind", ["tree", "chain", "any"])
@pytest.mark.parametrize("case", TREES, ids=[f"tree{i}" for i in range(len(TREES))])
def test_tree(case, kind):
    lens, lk, hq, hkv, d, page, dtype, layout, most = case
    c = Cache8(lk, hkv, d, page, seed=len(lens) + hq, layout=layout, spread=3.0)
    q = queries(sum(lens), hq, d, dtype, 7)
    if kind == "tree":
        masks = random_trees(lens, 3)
    elif kind == "any":
        # arbitrary bits, those past the tree among them; rows of none
        g = torch.Generator().manual_seed(9)
        masks = [int(torch.randint(0, 1 << 62, (1,), generator=g)) | (i & 1) << 63 for i in range(sum(lens))]
        masks[::3] = [0] * len(masks[::3])
    else:
        masks = None
    t = torch.tensor(bits_of(masks), dtype=torch.int64, device="cuda") if masks is not None else None
    o, lse = attn.attn_tree_fp8(q, *c.args(), cu_of(lens), tree_mask=t, max_tokens=most)
    ok()
    ref.check_attention(o, lse, q, c, lens, masks, 1.0 / math.sqrt(d))


def test_a_tree_of_one_token_is_a_decoding_step():
    lens = [400, 33, 1290]
    c = Cache8(lens, 2, 128, 16, 3)
    q = queries(3, 8, 128, BF, 1)
    a = attn.attn_decode_fp8(q, *c.args(), scale=0.3)
    b = attn.attn_tree_fp8(q, *c.args(), cu_of([1, 1, 1]), max_tokens=1, scale=0.3)
    ok()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_rows_behind_the_last_sequence_are_left():
    c = Cache8([50, 70], 2, 64, 16, 3)
    q = queries(9, 4, 64, HF, 1)
    out, lse = torch.full_like(q, 7.0), torch.full((4, 9), 7.0, device="cuda")
    attn.attn_tree_fp8(q, *c.args(), cu_of([3, 2]), out=out, lse=lse)
    ok()
    assert bool((out[5:] == 7.0).all()) and bool((lse[:, 5:] == 7.0).all())
    masks = [(2 << i) - 1 for n in (3, 2) for i in range(n)]
    ref.check_attention(out[:5], lse[:, :5], q[:5], c, [3, 2], masks, 0.125)


def test_offsets_that_do_not_begin_at_zero():
    c = Cache8([50, 70], 2, 64, 16, 3)
    q = queries(9, 4, 64, HF, 1)
    out = torch.full_like(q, 7.0)
    cu = torch.tensor([2, 5, 9], dtype=torch.int32, device="cuda")
    o, lse = attn.attn_tree_fp8(q, *c.args(), cu, out=out)
    ok()
    assert bool((out[:2] == 7.0).all())
    ref.check_attention(o[2:], lse[:, 2:], q[2:], c, [3, 4], None, 0.125)


def test_longer_trees_than_said_have_no_tokens():
    c = Cache8([50, 70, 30], 2, 64, 16, 3)
    q = queries(11, 4, 64, BF, 1)
    out = torch.full_like(q, 7.0)
    o, lse = attn.attn_tree_fp8(q, *c.args(), cu_of([3, 6, 2]), max_tokens=5, out=out)
    torch.cuda.synchronize()
    assert attn.get_error() == attn.ATTN_EDEVICE and attn.last_device_error() == attn.ATTN_DEVERR_BAD_SEQLENS
    assert bool((o[3:9] == 7.0).all())
    for lo, b, n in ((0, 0, 3), (9, 2, 2)):
        (k, ks), (v, vs) = c.rows(b, "k"), c.rows(b, "v")
        want = ref.attention(q[lo:lo + n], k, ks, v, vs, None, 0.125)[0]
        assert float((o[lo:lo + n].double() - want).abs().max()) < 0.02 * float(want.abs().max())


def test_bad_lengths_and_pages():
    c = Cache8([50, 70], 1, 64, 16, 3)
    q = queries(2, 2, 64, BF, 1)
    lens = torch.tensor([1 << 20, 70], dtype=torch.int32, device="cuda")
    o, lse = attn.attn_decode_fp8(q, c.k, c.v, c.ks, c.vs, c.table, lens)
    torch.cuda.synchronize()
    assert attn.get_error() == attn.ATTN_EDEVICE and attn.last_device_error() == attn.ATTN_DEVERR_BAD_SEQLENS
    assert bool((o[0] == 0).all()) and bool((lse[:, 0] == -math.inf).all())     # taken as having no keys
    table = c.table.clone()
    table[0, 2] = c.n_pages
    o, lse = attn.attn_decode_fp8(q, c.k, c.v, c.ks, c.vs, table, c.seqlens)
    torch.cuda.synchronize()
    assert attn.get_error() == attn.ATTN_EDEVICE and attn.last_device_error() == attn.ATTN_DEVERR_BAD_PAGE
    (k, ks), (v, vs) = c.rows(1, "k"), c.rows(1, "v")
    want = ref.attention(q[1:], k, ks, v, vs, None, 0.125)[0]
    assert float((o[1:].double() - want).abs().max()) < 0.02 * float(want.abs().max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["k", "v"])
def test_a_row_of_nan_reaches_what_sees_it_and_no_other(what, d):
    # key 100 (the third of the tree's four) is NaN: tokens 2 and 3 see it, 0 and 1 do not
    c = Cache8([102], 1, d, 16, 3)
    page, slot = c.places(0)
    (c.ks if what == "k" else c.vs)[page[100], slot[100]] = math.nan
    (c.k if what == "k" else c.v).view(torch.uint8)[page[100], slot[100]] = 0
    q = queries(4, 2, d, BF, 1)
    masks = torch.tensor([1, 3, 5, 13], device="cuda")
    o, lse = attn.attn_tree_fp8(q, *c.args(), cu_of([4]), tree_mask=masks)
    ok()
    assert bool(o[2:].isnan().all()) and not bool(o[:2].isnan().any())
    if what == "k":
        assert bool(lse[:, 2:].isnan().all())
    assert not bool(lse[:, :2].isnan().any())


def test_extreme_scales():
    # keys and values of very different sizes; the largest values on light keys
    lens = [700, 129]
    c = Cache8(lens, 2, 128, 16, 5, spread=20.0)
    q = queries(2, 8, 128, BF, 8)
    o, lse = attn.attn_decode_fp8(q, *c.args())
    ok()
    ref.check_attention(o, lse, q, c, [1, 1], None, 1.0 / math.sqrt(128))


def test_large_and_small_queries():
    c = Cache8([300, 140], 2, 64, 16, 5)
    for size in (2.0 ** -14, 40.0):
        q = (queries(2, 4, 64, HF, 8).float() * size).to(HF)
        o, lse = attn.attn_decode_fp8(q, *c.args())
        ok()
        ref.check_attention(o, lse, q, c, [1, 1], None, 0.125)
    q = torch.zeros(2, 4, 64, dtype=BF, device="cuda")
    o, lse = attn.attn_decode_fp8(q, *c.args())
    ok()
    ref.check_attention(o, lse, q, c, [1, 1], None, 0.125)
    q = queries(2, 4, 64, BF, 8)
    o, lse = attn.attn_decode_fp8(q, *c.args(), scale=0.0)
    ok()
    ref.check_attention(o, lse, q, c, [1, 1], None, 0.0)


def test_light_keys_reach_the_sum():
    # 65,535 keys of 2^-25 of the first's weight each are 2^-9 of the sum together
    n, d = 65536, 64
    c = Cache8([n], 1, d, 64, 5, poison=False)
    page, slot = c.places(0)
    k = torch.zeros(n, 1, d, device="cuda")
    k[0, 0, 0] = 1.0
    v = torch.ones(n, 1, d, device="cuda")
    v[0] = -1.0
    for pages, scales, x in ((c.k, c.ks, k), (c.v, c.vs, v)):
        x8, s = ref.quantise(x)
        pages.view(torch.uint8)[page, slot], scales[page, slot] = x8.view(torch.uint8), s
    q = torch.zeros(1, 1, d, dtype=HF, device="cuda")
    q[..., 0] = 25 * math.log(2.0)
    o, lse = attn.attn_decode_fp8(q, *c.args(), scale=1.0)
    ok()
    ref.check_attention(o, lse, q, c, [1], None, 1.0)


# ------------------------------------------------------------------ together, streams, graphs

def test_a_step_together():
    """Projection to answer: norms and rotation, append, tree attention over the cache,
    and the same attention by reading the cache back."""
    hq, hkv, d, lens, old = 8, 2, 128, [6, 1, 9], [300, 77, 0]
    total = sum(lens)
    c = Cache8([a + b for a, b in zip(old, lens)], hkv, d, 16, 5)
    qkv = queries(total, hq + 2 * hkv, d, BF, 3)
    q, k, v = qkv.split((hq, hkv, hkv), dim=1)
    w = torch.rand(2, d, generator=torch.Generator().manual_seed(1)).to(BF).cuda() + 0.5
    freqs, _ = attn.rotary_freqs(d)
    pos = torch.cat([torch.arange(a, a + b) for a, b in zip(old, lens)]).to(torch.int32).cuda()
    cu = cu_of(lens)
    qn, kn = attn.qk_norm_rotary(q, k, w[0], w[1], freqs, pos)
    attn.cache_append_fp8(kn, v, *c.args(), cu)
    o, lse = attn.attn_tree_fp8(qn, *c.args(), cu, max_tokens=9)
    ok()
    ref.check_attention(o, lse, qn, c, lens, None, 1.0 / math.sqrt(d))
    cu_k = cu_of([a + b for a, b in zip(old, lens)])
    kb, vb = attn.cache_read_fp8(*c.args(), cu_k, int(cu_k[-1]), BF)
    o2, lse2 = attn.attn_fwd(qn, kb, vb, causal=True, cu_seqlens=cu, cu_seqlens_k=cu_k)
    ok()
    # the same but for the 16-bit rounding of the keys and values read back
    assert float((o.float() - o2.float()).norm() / o.float().norm()) < 2.0 ** -6
    assert float((lse - lse2).abs().max()) < 2.0 ** -5


def run_all(c, q, k, v, cu, masks, freqs, outs, stream=None):
    attn.cache_append_fp8(k, v, *c.args(), cu, q=q, freqs=freqs, q_out=outs[0], stream=stream)
    attn.attn_tree_fp8(outs[0], *c.args(), cu, tree_mask=masks, max_tokens=40, out=outs[1], lse=outs[2], stream=stream)
    attn.cache_read_fp8(*c.args(), cu, outs[3].shape[0], BF, k_out=outs[3], v_out=outs[4], stream=stream)
    attn.attn_decode_fp8(outs[0][:len(c.lens)], *c.args(), out=outs[5], lse=outs[6], stream=stream)


def setting(d, seed):
    lens, lk, hq, hkv = [40, 7], [4000, 900], 8, 2
    c = Cache8(lk, hkv, d, 16, seed)
    q, k, v = queries(47, hq, d, BF, seed), queries(47, hkv, d, BF, seed + 1), queries(47, hkv, d, BF, seed + 2)
    masks = torch.tensor(bits_of(random_trees(lens, seed)), dtype=torch.int64, device="cuda")
    outs = [torch.empty_like(q), torch.empty_like(q), torch.empty(hq, 47, device="cuda"), torch.empty_like(k),
            torch.empty_like(v), torch.empty_like(q[:2]), torch.empty(hq, 2, device="cuda")]
    return (c, q, k, v, cu_of(lens), masks, attn.rotary_freqs(d)[0]), outs


def test_streams_graphs_and_repeats():
    sets = [setting(64, 1), setting(128, 2)]
    want = []
    for args, outs in sets:
        run_all(*args, outs)
        ok()
        want.append([t.clone() for t in outs])
    # again: the same bits; on other streams at once; from other threads at once
    for args, outs in sets:
        run_all(*args, outs)
    ok()
    assert all(torch.equal(a, b) for (_, outs), w in zip(sets, want) for a, b in zip(outs, w))
    streams = [torch.cuda.Stream() for _ in sets]
    for _, outs in sets:
        for t in outs:
            t.fill_(3)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (args, outs) in zip(streams, sets):
            run_all(*args, outs, stream=s)
    ok()
    assert all(torch.equal(a, b) for (_, outs), w in zip(sets, want) for a, b in zip(outs, w))

    def work(args, outs):
        for _ in range(5):
            run_all(*args, outs)

    threads = [threading.Thread(target=work, args=s) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ok()
    assert all(torch.equal(a, b) for (_, outs), w in zip(sets, want) for a, b in zip(outs, w))
    # two graphs, replayed side by side
    graphs = []
    for args, outs in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run_all(*args, outs)
        graphs.append(g)
    for _, outs in sets:
        for t in outs:
            t.fill_(5)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    ok()
    assert all(torch.equal(a, b) for (_, outs), w in zip(sets, want) for a, b in zip(outs, w))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [2, 16])
def test_many_short_sequences_repeat(hq, d):
    """Units of a few steps, several to a block: the join of the two groups of softmax
    warps at each unit's end."""
    lens = [(37 * i) % 900 for i in range(600)]
    c = Cache8(lens, 2, d, 64, 3)
    q = queries(len(lens), hq, d, BF, 4)
    want = attn.attn_decode_fp8(q, *c.args())
    ok()
    for _ in range(40):
        got = attn.attn_decode_fp8(q, *c.args())
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    ok()


def test_pages_whose_offsets_pass_32_bits():
    """The same rows at the far end of a pool of more than 4 GiB of keys, and in a small
    one: the same bits."""
    hkv, d, page, far, lens = 8, 128, 16, 266_000, [300, 17]
    assert far * page * hkv * d > 1 << 32
    f, _ = attn.rotary_freqs(d)
    q, k, v = (queries(sum(lens), h, d, BF, 6 + h) for h in (16, hkv, hkv))
    got = []
    for first in (0, far):
        n = first + 21
        pages = [torch.empty((n, page, hkv, d), dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
        scales = [torch.empty((n, page, hkv), device="cuda") for _ in range(2)]
        table = torch.full((2, 19), n - 1, dtype=torch.int32, device="cuda")
        table[0] += -torch.arange(19, dtype=torch.int32, device="cuda")
        table[1, :2] = torch.tensor([n - 21, n - 20], dtype=torch.int32)
        cache = (*pages, *scales, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
        qr = attn.cache_append_fp8(k, v, *cache, cu_of(lens), q=q, freqs=f)
        out = attn.cache_read_fp8(*cache, cu_of(lens), sum(lens))
        at = torch.tensor([lens[0] - 1, sum(lens) - 1], device="cuda")
        got.append((qr, *out, *attn.attn_decode_fp8(qr[at].contiguous(), *cache),
                    *attn.attn_tree_fp8(qr[at[1]:], *cache, torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda"))))
        ok()
        del pages, scales, cache
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_nothing_to_do():
    c = Cache8([20], 1, 64, 16, 1)
    e = torch.empty(0, 1, 64, dtype=BF, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    before = c.snapshot()
    attn.cache_append_fp8(e, e, *c.args(), cu)
    k, v = attn.cache_read_fp8(*c.args(), cu, 0)
    o, lse = attn.attn_tree_fp8(torch.empty(0, 2, 64, dtype=BF, device="cuda"), *c.args(), cu)
    ok()
    assert k.shape == v.shape == (0, 1, 64) and o.shape == (0, 2, 64) and lse.shape == (2, 0)
    assert torch.equal(c.k.view(torch.uint8), before[0])
