"""Calls over paged caches that are refused before anything reaches a GPU, and
scaled spectra of short contexts."""

import math

import pytest
import torch

from tiled_attention_attn_gb300 import attn

from .test_paged_boundary import evict


@pytest.mark.parametrize("w, n, wo, no, bad", [
    (4096, 64, 4096 + 512, 64, True),            # in the midst of the weights (2 x 2 rows of 64: 1,024 bytes)
    (4096, 64, 4096 + 1020, 8, True),            # their last entry
    (4096 + 124, 64, 4096, 8, True),             # an output (128 bytes) that reaches into them from below
    (4096 + 128, 64, 4096, 8, False),            # one that ends where they begin
    (4096, 64, 4096 + 4, 63, True),              # one entry further on
    (4096, 64, 4096 + 1024, 64, False),          # right behind them
    (4096 + 1024, 64, 4096, 64, False),          # right before them
    (4096, 64, 4096, 64, False),                 # the weights themselves
])
def test_eviction_weights_overlap(attn_lib, w, n, wo, no, bad):
    if not bad and torch.cuda.is_available():
        pytest.skip("accepted: the addresses are made up")
    rc = evict(attn_lib, w=w, n=n, wo=wo, no=no, kept=1 << 20, lens=1 << 21)
    assert (rc == attn.ATTN_EINVAL) == bad


@pytest.mark.parametrize("original", [1, 4, 6, 7, 40, 4096])
def test_yarn_of_short_contexts(original):
    # by the number of turns within the original context: below one f / factor, above 32 f
    plain, _ = attn.rotary_freqs(64)
    f, amp = attn.rotary_freqs(64, scaling="yarn", factor=8.0, original_len=original)
    assert abs(amp - (0.1 * math.log(8.0) + 1.0)) < 1e-15
    turns = plain * original / (2 * math.pi)
    assert torch.allclose(f[turns < 1.0] * 8.0, plain[turns < 1.0], rtol=1e-12)
    assert torch.equal(f[turns > 32.0], plain[turns > 32.0])
    assert bool((f <= plain).all()) and bool((f >= plain / 8.0 * (1 - 1e-12)).all())
