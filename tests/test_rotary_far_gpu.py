"""Scaled rotary embedding at far positions and large frequencies, against
angles in exact arithmetic; and frequencies that change under a gradient."""

import math

import pytest
import torch

from tiled_attention_attn_gb300 import attn

pytestmark = pytest.mark.gpu
HF = torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib(attn_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return attn_lib


def inverse_turn_bits(bits):
    """2^bits / (2 pi), rounded down: pi by Machin's formula in integers."""
    one = 1 << (2 * bits + 64)

    def arctan_of_inverse(x):
        term = total = one // x
        n, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total

    pi = 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))
    return (one << bits) // (2 * pi)


BITS = 300
INV_TURN = inverse_turn_bits(BITS)


def turned(pos, f):
    """cos and sin of pos * f: the angle's fraction of a turn in exact arithmetic."""
    num, den = float(f).as_integer_ratio()
    part = (pos * num * INV_TURN // den) % (1 << BITS)
    a = 2.0 * math.pi * (part / (1 << BITS))
    return math.cos(a), math.sin(a)


def check(y, pos, freqs):
    """y: rows of heads (1, 0) per pair.  Bar: half a step of the result (fp16;
    2^-25 below its normal range), the argument (2^-25 of a half turn from its
    rounding to fp32, 2^-31 from its 32 bits: 1.1e-7 rad), sine and cosine in
    fp32 (2^-22), the product."""
    half = len(freqs)
    got = y.double().cpu()
    for r, t in enumerate(pos):
        for i, f in enumerate(freqs):
            for g, want in zip((got[r, 0, i], got[r, 0, half + i]), turned(t, f)):
                bar = 2.0 ** -11 * abs(want) * 1.001 + 2.0 ** -25 + 2.0 ** -21
                assert abs(float(g) - want) <= bar, (t, f, float(g), want)


@pytest.mark.parametrize("freqs", [[1.0, 0.7498942093324559, 1e-4, 2.5e-5], [100.0, 37.7, 9.87654321, 1e3],
                                   [-100.0, -1e-4, -6.25, 1e9], [2.0 ** 40 + 0.3, 0.0, 3.0, -0.1]], ids=str)
def test_angles_at_far_positions(freqs):
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(1 << 30, (1 << 31) - 1, (600,), generator=g).tolist() + [(1 << 31) - 1, -(1 << 31), 0, 1]
    x = torch.zeros(len(pos), 1, 2 * len(freqs), dtype=HF, device="cuda")
    x[..., :len(freqs)] = 1.0
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    y = attn.rotary_scaled(x, torch.tensor(freqs, dtype=torch.float64), positions=p)
    torch.cuda.synchronize()
    check(y, pos, freqs)


def test_positions_that_offsets_carry_past_32_bits():
    f = [1.0, 0.1, 0.01, 0.001]
    x = torch.zeros(2, 5, 1, 8, dtype=HF, device="cuda")
    x[..., :4] = 1.0
    off = torch.tensor([(1 << 31) - 3, 7], dtype=torch.int32, device="cuda")
    y = attn.rotary_scaled(x, torch.tensor(f, dtype=torch.float64), offsets=off)
    z = attn.rotary_scaled(x.view(10, 1, 8), torch.tensor(f, dtype=torch.float64), offsets=off,
                           cu_seqlens=torch.tensor([0, 5, 10], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    pos = [(1 << 31) - 3 + i for i in range(5)] + [7 + i for i in range(5)]
    check(y.view(10, 1, 8), pos, f)
    assert torch.equal(z, y.view(10, 1, 8))


def test_frequencies_changed_before_the_backward_are_refused():
    f, a = attn.rotary_freqs(64)
    x = torch.randn(1, 8, 2, 64, generator=torch.Generator().manual_seed(1)).half().cuda().requires_grad_()
    y = attn.rotary_scaled_func(x, f, a)
    f.mul_(0.5)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()
    y = attn.rotary_scaled_func(x, f.tolist(), a)      # a sequence of numbers serves too
    y.sum().backward()
    want = attn.rotary_scaled(torch.ones_like(x), f, a, inverse=True)
    torch.cuda.synchronize()
    assert torch.equal(x.grad, want)
