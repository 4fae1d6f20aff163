"""Attention over caches of 8-bit floating point whose value rows differ in size by
many octaves: a row that a query does not see, or sees without weight, leaves its
output as it is, whatever the row's size; a row without a number reaches what sees
it, also where no other value row has one."""

import math

import pytest
import torch

from . import fp8_reference as ref
from .fp8_reference import Cache8, bits_of, cu_of
from .paged_reference import INF, half_step, score_error
from tiled_attention_attn_gb300 import attn

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib(attn_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.set_wait_timeout_ns(2_000_000_000)
    return attn_lib


def ok():
    torch.cuda.synchronize()
    assert attn.get_error() == attn.ATTN_OK, hex(attn.last_device_error())


def queries(n, hq, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, hq, d, generator=g).to(dtype).cuda()


def put(cache, b, key, which, x):
    """The row of one key, (Hkv, d), quantised into its place."""
    page, slot = (t[0] for t in cache.places(b, 1, key))
    pages, scales = (cache.k, cache.ks) if which == "k" else (cache.v, cache.vs)
    v8, s = ref.quantise(x.cuda())
    pages.view(torch.uint8)[page, slot] = v8.view(torch.uint8)
    scales[page, slot] = s


def bars(q, cols, k, ks, v, vs, masks, scale, weighty=None):
    """(O, lse, the bar of O, the bar of lse) of one sequence, cols tokens x heads to a
    key/value head at the most.  The bar of an element of O holds what its own row sees, by
    weight, and nothing else.  With a = sum p |v| / l, and t = max (p vs) sum |v| / l (v
    unscaled), p relative to the row's maximum:
    * its own rounding, half a step of |o| (fp16: 2^-25 where that is subnormal);
    * p vs, relative to the row's largest, is held times 2^7.  As rows of the products (more
      than 8 columns) in fp16, off by 2^-11 of it or an absolute 2^-25 2^-7, and the
      reference may lie four times above the largest: 2^-30 t.  As columns with the rest,
      times 2^11, in fp16 again: 2^-22 of it, or 2^-25 2^-11 2^-7: 2^-43 t;
    * a score off by ds moves p and l by ds each: 2 ds a.  ds: the products' sums in fp32
      (score_error), the query as e4m3 values, off by 2^-17.8 of its largest (sqrt(d)
      2^-17.8 max |q| |k| scale), and 2^-18 of exponentials, logarithms, sums and products
      in fp32.
    weighty: which keys can have weight (the norms of the others bound no weight's error)."""
    T, hq, d = q.shape
    want, lse, a, _ = ref.attention(q, k, ks, v, vs, masks, scale)
    kk = (k * ks[..., None]) if weighty is None else (k * ks[..., None])[weighty]
    ds = 2.0 ** -18 + score_error(q, kk, scale)
    ds += math.sqrt(d) * 2.0 ** -17.8 * float(q.abs().max()) * float(kk.double().norm(dim=-1).max()) * scale
    place = torch.arange(k.shape[0]) - (k.shape[0] - T)
    t = torch.zeros_like(a)
    for i in range(T):
        m = masks[i] if masks is not None else (2 << i) - 1
        tree = torch.tensor([bool(m >> x & 1) for x in range(T)])
        seen = torch.where(place < 0, torch.ones_like(tree[:1]).expand(place.shape[0]), tree[place.clamp(min=0)]).to(q.device)
        if not bool(seen.any()):
            continue
        for h in range(hq):
            g = h // (hq // k.shape[1])
            s = (k[seen, g].double() @ q[i, h].double()) * ks[seen, g].double() * scale
            p = (s - s.max()).exp()
            t[i, h] = (p * vs[seen, g].double()).max() * v[seen, g].double().abs().sum(0) / p.sum()
    rounding, floor = (2.0 ** -22, 2.0 ** -43) if cols <= 8 else (2.0 ** -11, 2.0 ** -30)
    bar = half_step(q.dtype) * want.abs() * 1.01 + (rounding + 2 * ds) * 1.01 * a + floor * t
    if q.dtype == HF:
        bar = bar + 2.0 ** -25
    return want, lse, bar, ds + 2.0 ** -20 + lse.abs() * 2.0 ** -22


def check(o, lse, q, cache, lens, masks, scale, cols, rows=None, weighty=None):
    """o and lse against the 64-bit form.  rows: which tokens of a sequence (all); weighty(b, k):
    as above."""
    at = 0
    for b, T in enumerate(lens):
        (k, ks), (v, vs) = cache.rows(b, "k"), cache.rows(b, "v")
        want, rl, bar, lbar = bars(q[at:at + T], cols, k, ks, v, vs, masks[at:at + T] if masks is not None else None, scale,
                                   None if weighty is None else weighty(k * ks[..., None]))
        mine = list(range(T)) if rows is None else rows
        err = (o[at:at + T].double() - want).abs()[mine]
        assert bool((err <= bar[mine]).all()), (b, float((err / bar[mine].clamp(min=1e-300)).max()))
        got = lse[:, at:at + T].double()
        assert torch.equal(got == -INF, rl == -INF)
        fin = rl != -INF
        assert bool(((got - rl).abs()[fin] <= lbar[fin]).all())
        at += T


# (head dimension, query heads of two key/value heads, tokens): the kernel with columns (up
# to 8 tokens x heads) and the one with rows
FORMS = [(64, 2, 2), (64, 4, 4), (128, 2, 5), (128, 8, 2), (64, 8, 8), (64, 16, 64), (128, 8, 12), (128, 12, 64)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("octaves", [0, 16, 24, 40, 110])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_a_large_value_row_that_is_not_seen(form, octaves, dtype):
    d, hq, T = form
    lens, lk = [T, T], [700, 3 * T]
    c = Cache8(lk, 2, d, 16, 3)
    g = torch.Generator().manual_seed(4)
    for b, n in enumerate(lk):
        put(c, b, n - T, "v", torch.randn(2, d, generator=g) * 2.0 ** octaves)
    # the first drafted token is the large row: siblings behind it see themselves and each
    # other as a chain, and not it; it sees itself
    masks = [(2 << i) - 1 - (1 if i else 0) for i in range(T)] * 2
    q = queries(2 * T, hq, d, dtype, 5)
    out = attn.attn_tree_fp8(q, *c.args(), cu_of(lens), max_tokens=T,
                             tree_mask=torch.tensor(bits_of(masks), dtype=torch.int64, device="cuda"))
    ok()
    # (the first token's own output is as large as its row: infinite in fp16 from 16 octaves on)
    rows = list(range(0 if dtype == BF or octaves == 0 else 1, T))
    for b in range(2):
        (k, ks), (v, vs) = c.rows(b, "k"), c.rows(b, "v")
        mine = slice(b * T, (b + 1) * T)
        want = ref.attention(q[mine], k, ks, v, vs, masks[mine], 1 / math.sqrt(d))[0]
        assert T == 1 or float(want[1:].abs().max()) < 64     # no part of the large row
    check(*out, q, c, lens, masks, 1 / math.sqrt(d), T * hq // 2, rows=rows)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("octaves", [16, 24, 40, 110])
@pytest.mark.parametrize("form", [(64, 2, 1), (128, 2, 1), (128, 8, 1), (64, 16, 1), (128, 32, 1), (128, 8, 9), (64, 4, 64)], ids=str)
def test_a_large_value_row_without_weight(form, octaves, dtype):
    d, hq, T = form
    lens, lk = [T, T, T], [200, 20000, 900]
    c = Cache8(lk, 2, d, 64, 6)
    g = torch.Generator().manual_seed(4)
    q = queries(3 * T, hq, d, dtype, 5)
    q[..., 0] = 4.0
    far = torch.zeros(2, d)
    far[:, 0] = -250.0 * math.sqrt(d)     # a score of -1000: no weight in 64 bits either
    for b, key in ((0, 3), (1, 0), (1, 9000), (2, 130)):
        put(c, b, key, "k", far)
        put(c, b, key, "v", torch.randn(2, d, generator=g) * 2.0 ** octaves)
    out = attn.attn_tree_fp8(q, *c.args(), cu_of(lens), max_tokens=T)
    ok()
    assert float(out[0].float().abs().max()) < 64
    check(*out, q, c, lens, None, 1 / math.sqrt(d), T * hq // 2, weighty=lambda kk: kk[:, 0, 0] > -100)


@pytest.mark.parametrize("form", [(64, 2, 1), (128, 8, 1), (128, 2, 8), (64, 4, 4)], ids=str)
@pytest.mark.parametrize("octaves", [16, 30])
def test_features_beside_a_large_one(octaves, form):
    """Half of the value rows have one feature of 2^octaves and zeros: the other features are
    made of the other rows alone."""
    d, hq, T = form
    n = 500
    c = Cache8([n], 2, d, 16, 6)
    g = torch.Generator().manual_seed(4)
    for key in range(0, n - T, 2):
        x = torch.zeros(2, d)
        x[:, 5] = torch.randn(2, generator=g) * 2.0 ** octaves
        put(c, 0, key, "v", x)
    q = queries(T, hq, d, BF, 5)
    o, lse = attn.attn_tree_fp8(q, *c.args(), cu_of([T]), max_tokens=T)
    ok()
    check(o, lse, q, c, [T], None, 1 / math.sqrt(d), T * hq // 2)


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -20, 2.0 ** 20, 2.0 ** 100])
@pytest.mark.parametrize("form", [(64, 2, 1), (128, 8, 1), (64, 16, 12), (128, 8, 64)], ids=str)
def test_values_of_any_one_size(form, size):
    d, hq, T = form
    c = Cache8([700], 2, d, 16, 6, spread=3.0)
    c.vs.mul_(size)
    q = queries(T, hq, d, BF, 5)
    o, lse = attn.attn_tree_fp8(q, *c.args(), cu_of([T]), max_tokens=T)
    ok()
    check(o, lse, q, c, [T], None, 1 / math.sqrt(d), T * hq // 2)


@pytest.mark.parametrize("octaves", [0, 60, 100])
@pytest.mark.parametrize("form", [(64, 2, 1), (128, 8, 1), (64, 16, 12), (128, 8, 64)], ids=str)
def test_rows_of_zeros_before_large_ones(form, octaves):
    """The reference of the first keys lies up to 189 octaves below that of the rest; their
    weights are in every sum."""
    d, hq, T = form
    n = 1500
    c = Cache8([n], 2, d, 16, 6)
    page, slot = c.places(0)
    c.vs[page, slot] *= 2.0 ** octaves
    c.vs[page[:700], slot[:700]] = 2.0 ** -126
    c.v.view(torch.uint8)[page[:700], slot[:700]] = 0
    q = queries(T, hq, d, BF, 5)
    o, lse = attn.attn_tree_fp8(q, *c.args(), cu_of([T]), max_tokens=T)
    ok()
    check(o, lse, q, c, [T], None, 1 / math.sqrt(d), T * hq // 2)


@pytest.mark.parametrize("form", [(64, 2, 1), (128, 8, 1), (64, 32, 1), (128, 8, 12)], ids=str)
@pytest.mark.parametrize("n, bad", [(1, (0, 1)), (40, (0, 40)), (128, (0, 64)), (128, (64, 128)), (256, (0, 128)),
                                    (512, (0, 256)), (512, (256, 512)), (20000, (0, 20000))])
def test_value_rows_without_a_number(form, n, bad):
    """All of the value rows that a warp, a group of warps or a block meets are NaN."""
    d, hq, T = form
    T = min(T, n)
    c = Cache8([n], 2, d, 16, 6)
    page, slot = (t[bad[0]:bad[1]] for t in c.places(0))
    c.vs[page, slot] = math.nan
    c.v.view(torch.uint8)[page, slot] = 0
    q = queries(T, hq, d, BF, 5)
    masks = torch.full((T,), -1, dtype=torch.int64, device="cuda")    # each sees all
    o, lse = attn.attn_tree_fp8(q, *c.args(), cu_of([T]), tree_mask=masks, max_tokens=T)
    ok()
    assert bool(o.isnan().all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("octaves", [0, 8, 13])
@pytest.mark.parametrize("form", [(64, 2, 1), (128, 8, 1), (64, 4, 4), (64, 32, 1), (128, 8, 9), (64, 16, 12)], ids=str)
def test_queries_with_one_large_feature(form, octaves, dtype):
    """Keys that are zero where the queries are large: the scores are made of the other
    features, which are all of one sign, so that what each loses adds up.  In the unit in
    which the largest is 2^8, a feature is 2^-5 or more here: in bf16 exact, as two values of
    4 or 3 bits.  In fp16 as e4m3, e4m3 and e5m2, what is left below e4m3's smallest step, at
    most 2^-10, keeps three bits: off by 2^-14, 2^-22 of the largest."""
    d, hq, T = form
    n, scale = 400, 1 / math.sqrt(d)
    c = Cache8([n], 2, d, 16, 6)
    g = torch.Generator().manual_seed(4)
    q = (1 + torch.rand(T, hq, d, generator=g)).to(dtype)
    q[..., 0] = 2.0 ** octaves
    k = (torch.rand(n, 2, 1, generator=g) * 8 / (1.5 * d * scale)).expand(-1, -1, d).clone()
    k[..., 0] = 0.0
    page, slot = c.places(0)
    k8, ks = ref.quantise(k.cuda())
    c.k.view(torch.uint8)[page, slot], c.ks[page, slot] = k8.view(torch.uint8), ks
    q = q.cuda()
    o, lse = attn.attn_tree_fp8(q, *c.args(), cu_of([T]), max_tokens=T)
    ok()
    (k, ks), (v, vs) = c.rows(0, "k"), c.rows(0, "v")
    small = q.clone()
    small[..., 0] = 0.0      # what the scores are made of
    want, rl, a, _ = ref.attention(small, k, ks, v, vs, None, scale)
    kk = k * ks[..., None]
    ds = 2.0 ** -18 + score_error(small, kk, scale)
    if dtype == HF:
        ds += 2.0 ** -22 * 2.0 ** max(octaves, 1) * float(kk.abs().double().sum(-1).max()) * scale
    bar = half_step(dtype) * want.abs() * 1.01 + (2.0 ** (-22 if T * hq <= 16 else -11) + 2 * ds) * 1.01 * a
    bar = bar + (2.0 ** -25 if dtype == HF else 1e-30)
    err = (o.double() - want).abs()
    assert bool((err <= bar).all()), float((err / bar).max())
    assert bool(((lse.double() - rl).abs() <= ds + 2.0 ** -20 + rl.abs() * 2.0 ** -22).all())
