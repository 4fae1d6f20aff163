"""The scratch memory that eager calls over a paged cache keep."""

import pytest
import torch

from .paged_reference import Cache, cu_of
from tiled_attention_attn_gb300 import attn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib(attn_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return attn_lib


class Calls:
    """The three calls that take scratch memory, on outputs of their own."""

    def __init__(self, d, seed):
        lens = [9000, 300]
        self.c = Cache(lens, 2, d, 16, BF, seed=seed)
        g = torch.Generator().manual_seed(seed)
        self.q1, self.q2 = (torch.randn(n, 8, d, generator=g).to(BF).cuda() for n in (2, 50))
        self.cu = cu_of([40, 10])
        self.o = [torch.empty_like(q) for q in (self.q1, self.q2)]
        self.lse = [torch.empty(8, q.shape[0], device="cuda") for q in (self.q1, self.q2)]
        self.w = torch.zeros(2, 2, self.c.table.shape[1] * 16, device="cuda")

    def __call__(self, stream=None):
        c = self.c
        attn.attn_decode_paged(self.q1, *c.args(), out=self.o[0], lse=self.lse[0], stream=stream)
        attn.attn_fwd_paged(self.q2, *c.args(), self.cu, out=self.o[1], lse=self.lse[1], stream=stream)
        attn.key_weights(self.q2, c.k, self.lse[1], c.table, c.seqlens, self.cu, decay=0.0, weights=self.w,
                         stream=stream)

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (*self.o, *self.lse, self.w)]


def allocations():
    return torch.cuda.memory_stats()["allocation.all.allocated"]


def test_repeated_calls_allocate_nothing():
    # both head dimensions, all three calls, on several streams, in turn
    calls = [Calls(64, 1), Calls(128, 2)]
    streams = [torch.cuda.Stream() for _ in range(3)]

    def round_():
        for s in streams:
            for f in calls:
                f(s)
            torch.cuda.synchronize()

    for _ in range(2):
        round_()
    want = [f.results() for f in calls]
    before = allocations()
    for _ in range(3):
        round_()
    assert allocations() == before
    for f, w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(f.results(), w))
    assert attn.get_error() == attn.ATTN_OK


def test_the_stream_used_last_keeps_its_memory():
    f = Calls(128, 1)
    hot, others = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(20)]
    for s in others:
        f(hot)
        f(s)
    torch.cuda.synchronize()
    before = allocations()
    f(hot)
    torch.cuda.synchronize()
    assert allocations() == before


def test_nothing_is_kept_for_streams_that_torch_does_not_own():
    # the handle of such a stream may come back as another stream's
    f = Calls(128, 1)
    f()
    want = f.results()
    inner = torch.cuda.Stream()
    s = torch.cuda.ExternalStream(inner.cuda_stream)
    for _ in range(3):
        s.wait_stream(torch.cuda.current_stream())
        before = allocations()
        f(s)
        assert allocations() == before + 3
        assert all(torch.equal(a, b) for a, b in zip(f.results(), want))
