"""The paged-cache operators at the ends of their ranges: 2^30 keys, thousands of
sequences, hundreds of heads, no queries at all."""

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
    attn.set_wait_timeout_ns(2_000_000_000)
    return attn_lib


def ok():
    torch.cuda.synchronize()
    assert attn.get_error() == attn.ATTN_OK, hex(attn.last_device_error())


def rand(*shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.fixture(scope="module")
def longest():
    """2^30 keys, less a few: a table of 2^22 entries that name five pages of 256."""
    n, page, d = (1 << 30) - 77, 256, 64
    k, v = rand(5, page, 1, d, dtype=BF, seed=1), rand(5, page, 1, d, dtype=BF, seed=2)
    table = torch.randint(0, 5, (1, 1 << 22), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    counts = torch.bincount(table[0, :-1].long(), minlength=5).double()[:, None].repeat(1, page)
    counts[int(table[0, -1]), : page - 77] += 1
    return n, k, v, table, torch.tensor([n], dtype=torch.int32, device="cuda"), counts.flatten()


def longest_form(q, k, v, counts, scale):
    """O, lse and each page slot's weight of one query over the counted slots, in 64 bits."""
    s = (q.double() @ k[:, :, 0].flatten(0, 1).double().t()) * scale        # (heads, slots)
    lse = (s.exp() * counts).sum(-1).log()
    p = (s - lse[:, None]).exp()
    vv = v[:, :, 0].flatten(0, 1).double()
    return (p * counts) @ vv, lse, p, (p * counts) @ vv.abs()


@pytest.mark.parametrize("decode", [True, False], ids=["decode", "chunk"])
def test_the_longest_cache(longest, decode):
    # bars as check_attention's and check_weights', and of sums of so many keys in
    # fp32: an accumulator takes up to 2^23 / 152 steps, 2^-23 each (5e-3 at worst)
    n, k, v, table, lens, counts = longest
    q = rand(1, 4, 64, dtype=BF, seed=4)
    scale, cu = 0.125, cu_of([1])
    if decode:
        o, lse = attn.attn_decode_paged(q, k, v, table, lens)
    else:
        o, lse = attn.attn_fwd_paged(q, k, v, table, lens, cu)
    ok()
    want, wl, p, a = longest_form(q[0], k, v, counts, scale)
    steps = (1 << 30) / 128 / 152 * 2.0 ** -23
    ds = ref.score_error(q, k[:, :, 0], scale) + 2.0 ** -18 + steps
    assert bool(((o[0].double() - want).abs() <= 2.0 ** -8 * (a + want.abs()) + 2 * ds * a).all())
    assert float((lse[:, 0].double() - wl).abs().max()) <= ds + 2.0 ** -18
    w = attn.key_weights(q, k, lse, table, lens, cu)
    ok()
    slot = table[0].long()[:, None] * 256 + torch.arange(256, device="cuda")
    at = torch.randint(0, n, (100_000,), generator=torch.Generator().manual_seed(5)).cuda()
    at[:3] = torch.tensor([0, n - 1, n - 2], device="cuda")
    r = p.sum(0)[slot.flatten()[at]]
    rel = 2 * ds + 2.0 ** -16
    assert bool(((w[0, 0][at].double() - r).abs() <= rel * r).all())
    assert bool((w[0, 0, n:] == 0).all())


def test_eviction_from_the_longest_cache(longest):
    n, k, v, table, lens, _ = longest
    w = torch.zeros(1, 1, 1 << 30, device="cuda")
    g = torch.Generator().manual_seed(6)
    heavy = torch.unique(torch.randint(0, n - 100, (3000,), generator=g))
    w[0, 0, heavy.cuda()] = 1.0
    budget, recent = 4000, 100
    dst = torch.arange(5, 21, dtype=torch.int32, device="cuda")[None]      # 16 pages of their own
    kp, vp = torch.zeros(21, 256, 1, 64, dtype=BF, device="cuda"), torch.zeros(21, 256, 1, 64, dtype=BF, device="cuda")
    kp[:5], vp[:5] = k, v
    kept, m, wout = attn.cache_evict(w, kp, vp, table, lens, budget, recent, dst_page_table=dst)
    ok()
    rest = budget - recent - heavy.numel()
    first = torch.tensor(sorted(set(range(rest + heavy.numel())) - set(heavy.tolist()))[:rest])
    want = torch.cat((torch.sort(torch.cat((heavy, first))).values, torch.arange(n - recent, n)))
    assert m.tolist() == [budget] and torch.equal(kept[0, 0].cpu().long(), want)
    assert torch.equal(wout[0, 0], w[0, 0, want.cuda()])
    src = table[0, want.cuda() // 256].long()
    for new, old in ((kp, k), (vp, v)):
        assert torch.equal(new[5:].flatten(0, 1)[:budget], old[src, want.cuda() % 256])


def test_thousands_of_sequences():
    lens = [(13 * i) % 70 for i in range(4000)]
    c = Cache(lens, 2, 64, 16, HF, seed=1, poison=False)
    new = [min(n, i % 3) for i, n in enumerate(lens)]
    q = rand(sum(new), 4, 64, dtype=HF, seed=2)
    o, lse = attn.attn_fwd_paged(q, *c.args(), cu_of(new))
    w = attn.key_weights(q, c.k, lse, c.table, c.seqlens, cu_of(new))
    ok()
    total = torch.zeros(4000, dtype=torch.float64, device="cuda")
    rows = torch.repeat_interleave(torch.arange(4000), torch.tensor(new)).cuda()
    total.index_add_(0, rows, torch.full((len(rows),), 4.0, dtype=torch.float64, device="cuda"))
    assert float((w.double().sum((1, 2)) - total).abs().max()) <= 1e-3     # each query's weights sum to 1
    k0, table = c.k.clone(), c.table.long()
    kept, m, _ = attn.cache_evict(w, c.k, c.v, c.table, c.seqlens, 20, 4)
    ok()
    assert m.tolist() == [min(n, 20) for n in lens]
    host_w, host_k = w.cpu(), kept.cpu()
    for b in range(0, 4000, 37):
        for g in range(2):
            want = ref.evict(host_w[b, g].tolist(), lens[b], 20, 4)
            assert host_k[b, g, :len(want)].tolist() == want
            j = torch.tensor(want, dtype=torch.long, device="cuda")
            i = torch.arange(len(want), device="cuda")
            assert torch.equal(c.k[table[b, i // 16], i % 16, g], k0[table[b, j // 16], j % 16, g])


@pytest.mark.parametrize("hkv", [151, 300])
def test_hundreds_of_heads(hkv):
    lens = [300, 17]
    c = Cache(lens, hkv, 64, 16, BF, seed=3)
    q = rand(2, 2 * hkv, 64, dtype=BF, seed=4)
    o, lse = attn.attn_decode_paged(q, *c.args())
    ok()
    ref.check_attention(o, lse, q, c, [1, 1], True, 0.125)
    w = attn.key_weights(q, c.k, lse, c.table, c.seqlens, cu_of([1, 1]))
    ok()
    for b in range(2):
        assert float((w[b].double().sum(-1) - 2.0).abs().max()) <= 1e-4


@pytest.mark.parametrize("decay", [0.5, 0.0])
def test_key_weights_of_no_queries(decay):
    # nothing is added: what was there decays
    c = Cache([300, 0, 17], 2, 128, 32, BF, seed=3)
    w = torch.rand(3, 2, 400, device="cuda")
    before = w.clone()
    q = torch.empty(0, 4, 128, dtype=BF, device="cuda")
    attn.key_weights(q, c.k, torch.empty(4, 0, device="cuda"), c.table, c.seqlens, cu_of([0, 0, 0]), decay=decay, weights=w)
    ok()
    for b, n in enumerate(c.lens):
        assert torch.equal(w[b, :, :n], before[b, :, :n] * decay) and torch.equal(w[b, :, n:], before[b, :, n:])
