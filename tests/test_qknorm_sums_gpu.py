"""The weights' gradients of the head norms over many tokens: every row of every head is in
the sums, whichever warp, turn of tokens or part of a token's heads it falls to."""

import math

import pytest
import torch

from .paged_reference import half_step
from .test_qknorm_gpu import Case
from tiled_attention_attn_gb300 import attn

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib(attn_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return attn_lib


def ok():
    torch.cuda.synchronize()
    assert attn.get_error() == attn.ATTN_OK


def depth(rows, heads, d):
    """Additions that a term passes through at the most: those of a thread, over the tokens
    of its warp (two blocks of 8 warps an SM, with fewer tokens one each; one more for the
    rest) and the heads that share its lanes' place; then over the lanes of a warp, the 8
    warps, every 32nd block, and a tree of 32."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lanes = 1 << max(0, math.ceil(math.log2(d // 16)))
    tokens = rows // (16 * sms) + 1
    return tokens * -(-heads // (32 // lanes)) + int(math.log2(32 // lanes)) + 8 + -(-2 * sms // 32) + 5


SIZES = [
    # rows, Hq, Hk, d
    (16384, 32, 8, 128),       # 6 tokens a warp, then parts of the rest
    (16421, 8, 8, 64),
    (2432, 16, 2, 128),        # a token each, where an SM pair of blocks has 16 warps and there are 152
    (2433, 5, 3, 128),
    (9001, 3, 1, 16),
    (5000, 12, 4, 448),
    (1537, 16, 16, 64),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows, hq, hk, d", SIZES)
def test_no_row_is_missing(rows, hq, hk, d, dtype):
    """dy = sign x: each term of dw is |z| > 0, so a row less is less by its share of the sum,
    which is above the bar: 2^-19 of each term (the sum of squares' 16 terms and 5 shuffles,
    the mean and eps, 23 roundings of 2^-24 that the root halves; rsqrt's 2 ulps, and two
    products: below 2^-19), and 2^-24 of the sum for each addition that a term passes
    through."""
    g = torch.Generator().manual_seed(rows + d)
    qkv = torch.randn(rows, hq + 2 * hk, d, generator=g).to(dtype).cuda()
    qkv[qkv.abs() < 0.25] = 0.25
    q, k, _ = qkv.split((hq, hk, hk), dim=1)
    w = torch.rand(2, d, generator=g).cuda() + 0.5
    dq, dk = q.sign().contiguous(), k.sign().contiguous()
    grads = attn.qk_norm_rotary_bwd(dq, dk, q, k, w[0], w[1], eps=1e-6)
    ok()
    for x, dw in ((q, grads[2]), (k, grads[3])):
        x = x.double()
        z = x.abs() / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        want = z.sum((0, 1))
        bar = want * (2.0 ** -19 + depth(rows, x.shape[1], d) * 2.0 ** -24)
        assert bool((z.sum(1).amin(0) > 2 * bar).all())
        err = (dw.double() - want).abs()
        assert bool((err <= bar).all()), float((err / bar).max())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows, hq, hk, d", SIZES)
def test_one_row_alone(rows, hq, hk, d, dtype):
    """All gradients but one head of one row are zero: dw is that head's g z, to fp32's
    rounding, wherever the row lies."""
    c = Case(rows, hq, hk, d, d, 1, False, dtype, F32)
    zero = [torch.zeros_like(t) for t in (c.dq, c.dk)]
    a, b = torch.randint(0, hq, (1,)).item(), hk - 1
    for row in sorted({0, 1, rows // 2, 2431 % rows, 2432 % rows, rows - 38 if rows > 38 else 0, rows - 2, rows - 1}):
        dq, dk = zero[0].clone(), zero[1].clone()
        dq[row, a], dk[row, b] = c.dq[row, a], c.dk[row, b]
        grads = attn.qk_norm_rotary_bwd(dq, dk, *c.args(), **c.kw())
        ok()
        one = Case(1, 1, 1, d, d, 1, False, dtype, F32)
        one.q, one.k, one.wq, one.wk, one.pos = c.q[row:row + 1, a:a + 1], c.k[row:row + 1, b:b + 1], c.wq, c.wk, c.pos[:, row:row + 1].contiguous()
        one.freqs, one.amplitude, one.dq, one.dk = c.freqs, c.amplitude, dq[row:row + 1, a:a + 1], dk[row:row + 1, b:b + 1]
        one.check_backward((grads[0][row:row + 1, a:a + 1], grads[1][row:row + 1, b:b + 1], *grads[2:]))
        for i, h in ((0, a), (1, b)):
            rest = grads[i].clone()
            rest[row, h] = 0
            assert not bool(rest.any())


def test_no_second_gradient():
    """The gradients have none of their own: asking for one is an error, not a wrong answer."""
    q = torch.randn(4, 2, 64, generator=torch.Generator().manual_seed(1)).to(BF).cuda().requires_grad_()
    y, _ = attn.qk_norm_rotary_func(q)
    (dq,) = torch.autograd.grad(y.float().square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        dq.float().sum().backward()
