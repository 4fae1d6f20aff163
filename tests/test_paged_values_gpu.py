"""Values at which the paged-cache operators can go wrong: queries left out of
the key weights, scores far from the ordinary, NaN in keys and queries that are
seen, many light keys, positions far out.  Tolerances are derived here or in
paged_reference."""

import math
from fractions import Fraction

import pytest
import torch

from . import paged_reference as ref
from .paged_reference import INF, Cache, cu_of
from tiled_attention_attn_gb300 import attn, paged

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib(attn_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.set_wait_timeout_ns(2_000_000_000)
    return attn_lib


def queries(lens, hq, d, dtype, seed):
    return torch.randn(sum(lens), hq, d, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def ok():
    torch.cuda.synchronize()
    assert attn.get_error() == attn.ATTN_OK, hex(attn.last_device_error())


# ---------------------------------------------------------------- key weights

def check_key_weights(w, q, c, lse, lq, causal, scale):
    """Bar, relative to the sum: the scores' error; lse / scale added to the
    score in fp32 (up to four truncated additions of a magnitude of |lse| +
    |score|, 2^-23 each); the exponential of a sum within 2^-22; m G additions."""
    at = 0
    for b, m in enumerate(lq):
        k = c.rows(c.k, b)
        lb = lse[:, at:at + m]
        r = ref.key_weights(q[at:at + m], k, lb, causal, scale)
        fin = lb[torch.isfinite(lb) & (lb.abs() < 1e30)]
        big = float(fin.abs().max()) if fin.numel() else 0.0
        ds = ref.score_error(q[at:at + m], k, scale) + big * 2.0 ** -21
        rel = math.expm1(2 * ds) + 2.0 ** -16 + m * (q.shape[1] // c.hkv) * 2.0 ** -24
        err = (w[b, :, :c.lens[b]].double() - r).abs()
        bar = rel * r + 2.0 ** -126
        assert bool((err <= bar).all()), (b, float((err / bar).max()))
        at += m


LEFT_OUT = [
    # new tokens, keys, Hq, Hkv, d, page, causal: tiles of 128 columns, of 16 (one token each), both forms of each
    ([300, 40], [500, 40], 8, 2, 128, 16, True),
    ([300, 130], [700, 300], 4, 4, 64, 32, False),
    ([1, 1, 1, 1, 1], [5, 129, 700, 3000, 260], 8, 2, 128, 16, True),
    ([1, 1, 1], [256, 2000, 17], 5, 1, 64, 64, False),
    ([40, 3], [9000, 300], 3, 1, 64, 64, True),
]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("value", [-INF, INF, 3.4e38])
@pytest.mark.parametrize("case", LEFT_OUT, ids=[f"case{i}" for i in range(len(LEFT_OUT))])
def test_queries_left_out_add_nothing(case, value, dtype):
    # lse = -inf leaves a query out, whatever the query holds; +inf and the
    # type's largest value give weights of zero by the formula
    lq, lk, hq, hkv, d, page, causal = case
    c = Cache(lk, hkv, d, page, dtype, seed=2)
    q = queries(lq, hq, d, dtype, 3)
    scale = 1.0 / math.sqrt(d)
    _, lse = attn.attn_fwd_paged(q, *c.args(), cu_of(lq), causal=causal)
    g = torch.Generator().manual_seed(5)
    out = (torch.rand(lse.shape, generator=g) < 0.3).cuda()
    out[:, 0] = True                       # all heads of a token
    out[0] |= torch.arange(lse.shape[1], device="cuda") % 2 == 0
    lse[out] = value
    given = q.clone()
    if value == -INF:
        given[out.t()] = torch.tensor([float("nan"), INF, -INF, 1.0], dtype=dtype, device="cuda").repeat(d // 4)
    w = attn.key_weights(given, c.k, lse, c.table, c.seqlens, cu_of(lq), causal=causal)
    ok()
    check_key_weights(w, q, c, lse, lq, causal, scale)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("scale, q_gain, k_gain", [(0.0, 1.0, 1.0), (2.0 ** -20, 1.0, 1.0), (2.0 ** -20, 1000.0, 20000.0),
                                                   (2.0 ** -10, 1.0, 1.0), (2.0 ** -10, 100.0, 300.0), (0.125, 8.0, 8.0),
                                                   (2.0, 1.0, 1.0), (2.0, 3.0, 4.0)])
@pytest.mark.parametrize("lq, lk", [([200, 30], [300, 500]), ([1, 1], [300, 500])], ids=["chunk", "decode"])
def test_key_weights_of_any_scale(lq, lk, scale, q_gain, k_gain, dtype):
    # scale 0 (no products), the smallest scale, |lse| into the hundreds and
    # |lse / scale| past 4e8
    c = Cache(lk, 2, 64, 16, dtype, seed=6)
    c.k.mul_(k_gain).clamp_(-60000.0, 60000.0)   # (finite in fp16: 20000 x 3.3 would not be)
    q = queries(lq, 6, 64, dtype, 7) * q_gain
    _, lse = attn.attn_fwd_paged(q, *c.args(), cu_of(lq), scale=scale)
    w = attn.key_weights(q, c.k, lse, c.table, c.seqlens, cu_of(lq), scale=scale)
    ok()
    check_key_weights(w, q, c, lse, lq, True, scale)


# ---------------------------------------------------------------- NaN that is seen

def where_key(c, b, j):
    return int(c.table[b, j // c.page]), j % c.page


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n, j", [(60, 3), (700, 699), (40000, 5), (40000, 39990)])
def test_nan_reaches_every_query_that_sees_it(n, j, d, dtype):
    """A NaN in a key makes O and lse of the queries that see it NaN, as the
    formula does, also where the cache is cut into pieces; nothing else."""
    nan = float("nan")
    c = Cache([n, 300], 2, d, 16, dtype, seed=4)
    q1, q2, cu = queries([1, 1], 8, d, dtype, 5), queries([20, 9], 8, d, dtype, 6), cu_of([20, 9])
    want1, want2 = attn.attn_decode_paged(q1, *c.args()), attn.attn_fwd_paged(q2, *c.args(), cu)
    page, slot = where_key(c, 0, j)
    c.k[page, slot, 0] = nan                       # the first head's key
    o, lse = attn.attn_decode_paged(q1, *c.args())
    ok()
    assert bool(o[0, :4].isnan().all()) and bool(lse[:4, 0].isnan().all())
    keep = torch.ones(2, 8, dtype=torch.bool, device="cuda")
    keep[0, :4] = False
    assert torch.equal(o[keep], want1[0][keep]) and torch.equal(lse.t()[keep], want1[1].t()[keep])
    o, lse = attn.attn_fwd_paged(q2, *c.args(), cu)
    ok()
    sees = torch.arange(20, device="cuda") >= j - (n - 20)
    gone = torch.zeros(29, 8, dtype=torch.bool, device="cuda")
    gone[:20, :4] = sees[:, None]
    assert bool(o[gone].isnan().all()) and bool(lse.t()[gone].isnan().all())
    assert torch.equal(o[~gone], want2[0][~gone]) and torch.equal(lse.t()[~gone], want2[1].t()[~gone])


@pytest.mark.parametrize("n", [60, 40000])
def test_nan_in_a_query(n):
    c = Cache([n, 300], 2, 128, 16, BF, seed=4)
    q1, q2, cu = queries([1, 1], 8, 128, BF, 5), queries([20, 9], 8, 128, BF, 6), cu_of([20, 9])
    want1, want2 = attn.attn_decode_paged(q1, *c.args()), attn.attn_fwd_paged(q2, *c.args(), cu)
    q1[0, 3, 70] = q2[4, 5, 0] = float("nan")
    for q, (o0, l0), (o, lse) in ((q1, want1, attn.attn_decode_paged(q1, *c.args())),
                                  (q2, want2, attn.attn_fwd_paged(q2, *c.args(), cu))):
        ok()
        gone = q.isnan().any(-1)
        assert bool(o[gone].isnan().all()) and bool(lse.t()[gone].isnan().all())
        assert torch.equal(o[~gone], o0[~gone]) and torch.equal(lse.t()[~gone], l0.t()[~gone])


# ---------------------------------------------------------------- many light keys

@pytest.mark.parametrize("heavy", [0.0, 1.0])
@pytest.mark.parametrize("decode", [True, False], ids=["decode", "chunk"])
@pytest.mark.parametrize("d", [64, 128])
def test_many_light_keys_count_in_fp16(d, decode, heavy):
    """One heavy key of value `heavy` before 65,535 of value 1 and weight e^-17.5
    (2^-25.2) each, 1.6e-3 of the sum together: O = (heavy + light) / (1 + light).
    Sequences (all on the same pages) or queries so many that no unit is cut.
    Bar of O: its rounding, half a step (2^-11 of it); of a weight half a step too,
    or, below the normal range, 2^-32 of the largest; and of u, which the tensor
    core accumulates key by key in fp32, truncating, 2^-23 of its magnitude a key
    (with heavy = 1 that alone is 8e-3: products so far below u are not in its
    reach)."""
    n, page, light = 65536, 64, 17.5
    k = torch.zeros(n // page, page, 1, d, dtype=HF, device="cuda")
    k[0, 0, 0, 0] = light
    v = torch.ones_like(k)
    v[0, 0] = heavy
    scale = 1.0 / math.sqrt(d)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None]
    B, m = (2 * sms, 1) if decode else (1, 256 * sms)
    q = torch.zeros(B * m, 1, d, dtype=HF, device="cuda")
    q[..., 0] = 1.0 / scale
    top = light * float(q[0, 0, 0]) * scale
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    table = table.repeat(B, 1)
    if decode:
        o, lse = attn.attn_decode_paged(q, k, v, table, lens)
    else:
        o, lse = attn.attn_fwd_paged(q, k, v, table, lens, cu_of([m]), causal=False)
    ok()
    light_sum = (n - 1) * math.exp(-top)
    total = 1.0 + light_sum
    want = (heavy + light_sum) / total
    bar = 2.0 ** -11 * (want + heavy) + n * 2.0 ** -32 + want * n * 2.0 ** -23 + 2.0 ** -25
    # the sum of exponentials: a thread adds up to n / 128 + 128 terms or partial
    # sums in fp32 to one that stays about the total, each addition off by up to
    # 2^-24 of it (a weight of 2^-25.2 beside 1 is lost in one)
    sums = (n / 128 + 128) * 2.0 ** -24
    assert float((o.double() - want).abs().max()) <= bar + want * sums
    assert heavy or light_sum > 20 * bar        # (what is at stake is well above the bar)
    assert float((lse.double() - (top + math.log(total))).abs().max()) <= top * 2.0 ** -22 + 2.0 ** -18 + sums
