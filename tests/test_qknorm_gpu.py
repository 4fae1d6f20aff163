"""Norms of heads with rotary embedding, forward and backward, against their
64-bit forms: head sizes, axes, pairings, strides, weights, lengths from none to
many; gradients against the formula's and against differences.

Tolerances.  With z = x r, every fp32 step is off by 2^-24 of its result: the sum
of squares (16 terms and up to 5 shuffles: 21), rsqrt (2 ulps), three products,
sine and cosine (2^-23, and 2^-23 from the argument) and the pair's two products
and their sum: below 64 steps, 2^-18 of the pair's magnitudes in all.  The output
is rounded once: half a step of it (in fp16 2^-25 where it is subnormal)."""

import math
import threading

import pytest
import torch

from .paged_reference import half_step
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


def pairs(rot, inter, dev):
    p = torch.arange(rot // 2, device=dev)
    return (2 * p, 2 * p + 1) if inter else (p, p + rot // 2)


def turned(x, angle, rot, inter, amplitude, sign=1.0):
    y = x.clone()
    a, b = pairs(rot, inter, x.device)
    c, s = (angle.cos() * amplitude)[:, None], (angle.sin() * amplitude * sign)[:, None]
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def magnitude(x, rot, inter, amplitude):
    """For each feature, the sum of its pair's magnitudes times the amplitude."""
    y = x.abs().clone()
    a, b = pairs(rot, inter, x.device)
    y[..., a] = y[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(amplitude)
    return y


def forward(x, w, angle, rot, inter, amplitude, eps):
    z = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return turned(z * w, angle, rot, inter, amplitude)


class Case:
    def __init__(self, rows, hq, hk, d, rot, axes, inter, dtype, wtype, scaling="yarn", seed=0, strided=True, far=1 << 20):
        g = torch.Generator().manual_seed(seed + rows + d)
        self.hq, self.hk, self.d, self.rot, self.inter, self.dtype, self.eps = hq, hk, d, rot, inter, dtype, 1e-5
        qkv = (torch.randn(rows, hq + 2 * hk, d, generator=g) * 3).to(dtype).cuda()
        self.q = qkv[:, :hq] if strided else qkv[:, :hq].contiguous()
        self.k = None if hk == 0 else qkv[:, hq:hq + hk] if strided else qkv[:, hq:hq + hk].contiguous()
        self.wq, self.wk = ((torch.randn(d, generator=g) * 0.5 + 1).to(wtype).cuda() if wtype and h else None
                            for h in (hq, hk))
        self.freqs, self.amplitude = attn.rotary_freqs(rot, scaling=scaling, factor=8.0) if rot else (None, 1.0)
        self.axes = [int(a) for a in torch.randint(0, axes, (rot // 2,), generator=g)] if axes > 1 else None
        self.pos = torch.randint(-far, far, (axes, rows), generator=g).to(torch.int32).cuda() if rot else None
        self.dq, self.dk = (torch.randn(rows, h, d, generator=g).to(dtype).cuda() if h else None for h in (hq, hk))

    def angle(self):
        if not self.rot:
            return torch.zeros(self.q.shape[0], 0, dtype=torch.float64, device="cuda")
        a = torch.tensor(self.axes or [0] * (self.rot // 2), device="cuda")
        return self.pos.double()[a].t() * self.freqs.cuda()

    def args(self):
        return self.q, self.k, self.wq, self.wk, self.freqs, self.pos

    def kw(self):
        return dict(axes=self.axes, eps=self.eps, amplitude=self.amplitude, interleaved=self.inter)

    def sides(self):
        return [s for s in ((self.q, self.wq, self.dq), (self.k, self.wk, self.dk)) if s[0] is not None]

    def weight(self, w):
        return torch.ones(self.d, dtype=torch.float64, device="cuda") if w is None else w.double()

    def check_forward(self, outs):
        for (x, w, _), y in zip(self.sides(), outs):
            x, w = x.double(), self.weight(w)
            want = forward(x, w, self.angle(), self.rot, self.inter, self.amplitude, self.eps)
            z = x / torch.sqrt((x * x).mean(-1, keepdim=True) + self.eps) * w
            bar = half_step(self.dtype) * want.abs() * 1.001 + 2.0 ** -18 * magnitude(z, self.rot, self.inter, self.amplitude)
            if self.dtype == HF:
                bar = bar + 2.0 ** -25
            err = (y.double() - want).abs()
            assert y.is_contiguous() and bool((err <= bar).all()), float((err / bar.clamp(min=1e-30)).max())

    def check_backward(self, grads):
        """dx = r (g w - z mean(g w z)): its terms are off by 2^-18 of their magnitudes
        (the mean's sum has d terms: 2^-18 of the sum of magnitudes).  dw sums rows x
        heads terms, each off by 2^-18 of its magnitude, with fp32 additions, at most
        one per term."""
        dx, dw = grads[:2], grads[2:]
        for i, (x, w, dy) in enumerate(self.sides()):
            x, w64, dy = x.double(), self.weight(w), dy.double()
            r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + self.eps)
            z, g = x * r, turned(dy, self.angle(), self.rot, self.inter, self.amplitude, -1.0)
            big = magnitude(dy, self.rot, self.inter, self.amplitude)
            m = (g * w64 * z).mean(-1, keepdim=True)
            want = r * (g * w64 - z * m)
            slack = r * (big * w64.abs() + z.abs() * (big * (w64 * z).abs()).mean(-1, keepdim=True))
            bar = half_step(self.dtype) * want.abs() * 1.001 + 2.0 ** -17 * slack
            if self.dtype == HF:
                bar = bar + 2.0 ** -25
            err = (dx[i].double() - want).abs()
            assert bool((err <= bar).all()), float((err / bar.clamp(min=1e-30)).max())
            if w is None:
                assert dw[i] is None
                continue
            want = (g * z).sum((0, 1))
            n = x.shape[0] * x.shape[1]
            bar = (2.0 ** -18 + n * 2.0 ** -24) * (big * z.abs()).sum((0, 1)) + half_step(w.dtype) * want.abs() * 1.001 + 1e-30
            if w.dtype == HF:
                bar = bar + 2.0 ** -25
            err = (dw[i].double() - want).abs()
            assert dw[i].dtype == w.dtype and bool((err <= bar).all()), float((err / bar).max())


CASES = [
    # rows, Hq, Hk, d, rot, axes, interleaved, dtype, weights' dtype
    (1, 1, 1, 64, 64, 1, False, BF, BF),
    (1, 32, 8, 128, 128, 1, False, BF, F32),
    (7, 5, 3, 64, 32, 2, True, HF, HF),
    (33, 16, 2, 128, 128, 3, False, BF, BF),
    (130, 12, 12, 128, 64, 4, True, HF, F32),
    (1000, 8, 1, 64, 64, 3, True, BF, BF),
    (3000, 16, 4, 128, 128, 1, False, HF, HF),
    (2, 3, 1, 16, 16, 1, False, BF, BF),
    (19, 7, 2, 32, 16, 8, True, BF, BF),
    (65, 4, 2, 96, 96, 3, False, HF, HF),
    (40, 9, 3, 80, 48, 2, True, BF, BF),
    (51, 4, 4, 256, 128, 2, False, BF, BF),
    (23, 3, 2, 512, 512, 3, False, HF, F32),
    (9, 2, 1, 496, 240, 2, True, BF, BF),
    (77, 71, 0, 128, 128, 1, False, BF, BF),        # queries alone
    (45, 8, 2, 128, 0, 1, False, BF, BF),           # norms alone
    (45, 8, 2, 64, 64, 1, False, HF, None),         # no weights
    (0, 8, 2, 128, 128, 1, False, BF, BF),
]


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[f"case{i}" for i in range(len(CASES))])
def test_forward_and_backward(case, strided):
    c = Case(*case, strided=strided)
    outs = attn.qk_norm_rotary(*c.args(), **c.kw())
    ok()
    c.check_forward(outs)
    assert (outs[1] is None) == (c.k is None)
    grads = attn.qk_norm_rotary_bwd(c.dq, c.dk, *c.args(), **c.kw())
    ok()
    c.check_backward(grads)
    again = attn.qk_norm_rotary_bwd(c.dq, c.dk, *c.args(), **c.kw())
    ok()
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(grads, again))


def test_one_axis_with_and_without_its_axis():
    c = Case(50, 4, 2, 64, 64, 1, False, BF, BF)
    a = attn.qk_norm_rotary(*c.args(), **c.kw())
    b = attn.qk_norm_rotary(c.q, c.k, c.wq, c.wk, c.freqs, c.pos[0], **c.kw())
    both = torch.stack((c.pos[0], torch.zeros_like(c.pos[0])))
    d = attn.qk_norm_rotary(c.q, c.k, c.wq, c.wk, c.freqs, both, **{**c.kw(), "axes": [0] * 32})
    ok()
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and all(torch.equal(x, y) for x, y in zip(a, d))


def test_the_rotation_is_that_of_rotary_scaled():
    # positions across the whole range; unit weights
    c = Case(200, 4, 2, 64, 64, 1, True, BF, None, far=(1 << 31) - 1)
    y, _ = attn.qk_norm_rotary(*c.args(), **c.kw())
    n, _ = attn.qk_norm_rotary(c.q, eps=c.eps)
    z = attn.rotary_scaled(n, c.freqs, c.amplitude, interleaved=True, positions=c.pos[0])
    ok()
    c.check_forward((y,))
    # z has been rounded once more, before the rotation
    assert float((y.double() - z.double()).norm() / y.double().norm()) < 2.0 ** -8


def test_batches_in_place_and_outputs():
    c = Case(6 * 50, 4, 2, 128, 128, 2, False, HF, HF, strided=False)
    want = attn.qk_norm_rotary(*c.args(), **c.kw())
    q4, k4, pos = c.q.view(6, 50, 4, 128), c.k.view(6, 50, 2, 128), c.pos.view(2, 6, 50)
    got = attn.qk_norm_rotary(q4, k4, c.wq, c.wk, c.freqs, pos, **c.kw())
    assert got[0].shape == q4.shape and all(torch.equal(a.view_as(b), b) for a, b in zip(got, want))
    # a batch of slices of one projection
    fused = torch.cat((q4, k4), dim=2)
    got = attn.qk_norm_rotary(fused[:, :, :4], fused[:, :, 4:], c.wq, c.wk, c.freqs, pos, **c.kw())
    assert all(torch.equal(a.view_as(b), b) for a, b in zip(got, want))
    # heads before tokens
    qh = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    got = attn.qk_norm_rotary(qh, c.k, c.wq, c.wk, c.freqs, c.pos, **c.kw())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    grads = attn.qk_norm_rotary_bwd(c.dq, c.dk, *c.args(), **c.kw())
    dq, dk = c.dq.clone(), c.dk.clone()
    mine = attn.qk_norm_rotary_bwd(dq, dk, *c.args(), **c.kw(), dq=dq, dk=dk)
    assert mine[0] is dq and all(torch.equal(a, b) for a, b in zip(mine, grads))
    q, k = c.q.clone(), c.k.clone()
    got = attn.qk_norm_rotary(q, k, c.wq, c.wk, c.freqs, c.pos, **c.kw(), q_out=q, k_out=k)
    ok()
    assert got[0] is q and all(torch.equal(a, b) for a, b in zip(got, want))


def test_outputs_that_overlap_inputs_are_refused():
    buf = torch.zeros(40 * 4 * 64 + 64, dtype=BF, device="cuda")
    q = buf[:40 * 4 * 64].view(40, 4, 64)
    for out in (buf[64:].view(40, 4, 64),):
        with pytest.raises(attn.AttnError):
            attn.qk_norm_rotary(q, q_out=out)
    qk = torch.zeros(40, 6, 64, dtype=BF, device="cuda")
    with pytest.raises(attn.AttnError):
        attn.qk_norm_rotary(qk[:, :4], qk[:, 4:], k_out=qk.view(-1)[:40 * 2 * 64].view(40, 2, 64))


def test_zeros_large_values_and_not_finite_ones():
    x = torch.zeros(6, 2, 64, dtype=BF, device="cuda")
    x[1] = 1e-20
    x[2] = 1e18
    x[3, 0, 5] = math.nan
    x[4, 1, 0] = math.inf
    x[5] = torch.randn(2, 64)
    y, _ = attn.qk_norm_rotary(x, eps=1e-6)
    ok()
    assert bool((y[0] == 0).all()) and torch.allclose(y[1].float(), x[1].float() * 1e3, rtol=2.0 ** -7)
    assert bool((y[2] == 1).all())
    assert bool(y[3, 0].isnan().all()) and not bool(y[3, 1].isnan().any())
    assert bool(y[4, 1, 0].isnan()) and bool((y[4, 1, 1:] == 0).all()) and bool((y[4, 0] == 0).all())
    assert bool(torch.isfinite(y[5].float()).all())


@pytest.mark.parametrize("dtype", [BF, HF])
def test_autograd(dtype):
    c = Case(60, 6, 2, 64, 32, 2, True, dtype, F32)
    leaves = [t.detach().clone().requires_grad_() for t in (c.q, c.k, c.wq, c.wk)]
    q, k = attn.qk_norm_rotary_func(*leaves, c.freqs, c.pos, **c.kw())
    c.check_forward((q, k))
    torch.autograd.backward((q, k), (c.dq, c.dk))
    ok()
    c.check_backward([t.grad for t in leaves])
    # one output used, one leaf wanted, a gradient that is an expanded one
    leaves = [t.detach().clone() for t in (c.q, c.k, c.wq, c.wk)]
    leaves[1].requires_grad_()
    k = attn.qk_norm_rotary_func(*leaves, c.freqs, c.pos, **c.kw())[1]
    k.sum().backward()
    ok()
    want = attn.qk_norm_rotary_bwd(torch.zeros_like(c.dq), torch.ones_like(c.dk), *c.args(), **c.kw())[1]
    assert torch.equal(leaves[1].grad, want)


def test_gradients_against_differences():
    """The change of L = sum(dy y) along a random direction, by central differences of
    the 64-bit forward, against the kernel's gradients: each of them is off by half
    a step (2^-11 of it) and 2^-17 of its terms, so their sum by sum |error| |direction|,
    the differences by h^2 times the third derivative (h = 1e-4: below 1e-6 of it)."""
    c = Case(20, 3, 2, 64, 64, 2, False, HF, F32, scaling=None)
    dq, dk, dwq, dwk = attn.qk_norm_rotary_bwd(c.dq, c.dk, *c.args(), **c.kw())
    ok()
    g = torch.Generator().manual_seed(5)
    for (x, w, dy), dx, dw in zip(c.sides(), (dq, dk), (dwq, dwk)):
        vx, vw = (torch.randn(t.shape, generator=g).double().cuda() for t in (x, w))

        def loss(t):
            return (forward(x.double() + t * vx, w.double() + t * vw, c.angle(), c.rot, c.inter, c.amplitude, c.eps) * dy.double()).sum()

        h = 1e-4
        slope = float((loss(h) - loss(-h)) / (2 * h))
        mine = float((dx.double() * vx).sum() + (dw.double() * vw).sum())
        bar = float((dx.double().abs() * vx.abs()).sum()) * 2.0 ** -10 + float((dw.double().abs() * vw.abs()).sum()) * 2.0 ** -12
        assert abs(slope - mine) <= bar + 1e-5 * abs(slope), (slope, mine, bar)


def test_changed_positions_before_the_backward_are_an_error():
    c = Case(30, 4, 2, 64, 64, 1, False, BF, BF)
    q = c.q.detach().clone().requires_grad_()
    y, _ = attn.qk_norm_rotary_func(q, c.k, c.wq, c.wk, c.freqs, c.pos, **c.kw())
    c.pos.add_(1)
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_streams_graphs_and_threads():
    sets = [Case(900, 8, 2, 128, 128, 3, False, BF, BF), Case(901, 6, 6, 64, 32, 1, True, BF, BF)]
    want = [attn.qk_norm_rotary_bwd(c.dq, c.dk, *c.args(), **c.kw()) for c in sets]
    ok()
    got = [None, None]

    def work(i, stream):
        for _ in range(5):
            got[i] = attn.qk_norm_rotary_bwd(sets[i].dq, sets[i].dk, *sets[i].args(), **sets[i].kw(), stream=stream)

    streams = [torch.cuda.Stream() for _ in sets]
    for s in (streams, [None, None]):
        threads = [threading.Thread(target=work, args=(i, s[i])) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        ok()
        assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
    # two graphs of forward and backward, replayed side by side; new inputs in the same places
    graphs = []
    for c in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = (*attn.qk_norm_rotary(*c.args(), **c.kw()), *attn.qk_norm_rotary_bwd(c.dq, c.dk, *c.args(), **c.kw()))
        graphs.append((g, out))
    for c in sets:
        c.q.mul_(0.5)
        c.dk.add_(1)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    ok()
    for c, (_, out) in zip(sets, graphs):
        c.check_forward(out[:2])
        c.check_backward(out[2:])


def test_rows_whose_offsets_pass_32_bits():
    rows, h, d, tail = 525_000, 32, 128, 500
    assert rows * h * d > 1 << 31
    q, g = (torch.randn(rows, h, d, dtype=BF, device="cuda") for _ in range(2))
    w = torch.randn(d, device="cuda")
    f, _ = attn.rotary_freqs(d)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    y = attn.qk_norm_rotary(q, q_weight=w, freqs=f, positions=pos)[0]
    dq = attn.qk_norm_rotary_bwd(g, None, q, q_weight=w, freqs=f, positions=pos)[0]
    at = slice(rows - tail, rows)
    assert torch.equal(y[at], attn.qk_norm_rotary(q[at], q_weight=w, freqs=f, positions=pos[at])[0])
    assert torch.equal(dq[at], attn.qk_norm_rotary_bwd(g[at], None, q[at], q_weight=w, freqs=f, positions=pos[at])[0])
    ok()


def test_a_captured_training_step():
    c = Case(300, 8, 2, 128, 64, 3, False, BF, F32)
    leaves = [t.clone().requires_grad_() for t in c.args()[:4]]

    def step():
        y = attn.qk_norm_rotary_func(*leaves, *c.args()[4:], **c.kw())
        torch.autograd.backward(y, (c.dq, c.dk))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for t in leaves:
        t.grad = None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    c.q.mul_(0.5)
    with torch.no_grad():
        leaves[0].copy_(c.q)
    for _ in range(2):
        g.replay()
    ok()
    want = attn.qk_norm_rotary_bwd(c.dq, c.dk, *c.args(), **c.kw())
    assert all(torch.equal(t.grad, w) for t, w in zip(leaves, want))
