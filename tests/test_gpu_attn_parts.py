"""Attention over the cache where one request's keys are spread over many CTAs:
every CTA adds up its share of the rows, or the last one all of them."""
import pytest
import torch

from speculative_decoding_pe_gb300 import _native
from test_gpu_attn import BF, HEADS, Cached, draft

pytestmark = pytest.mark.gpu


def requests(kind, lengths):
    return [[n] if kind == "token" else draft(n, n % 8) for n in lengths]


def counters(c):
    return c.ws[:4096]


@pytest.mark.parametrize("Hq, Hkv, D", HEADS)
@pytest.mark.parametrize("kind", ["token", "draft"])
@pytest.mark.parametrize("lengths", [[2047], [2300, 1], [9000, 60, 5001], [700] * 3])
def test_parts_add_up(Hq, Hkv, D, kind, lengths):
    c = Cached(requests(kind, lengths), Hq, Hkv, D, 16, 11, uniform=True, extra=200)
    c.check()
    assert not counters(c).any()


@pytest.mark.parametrize("kind", ["token", "draft"])
def test_one_request_of_one_head_over_every_cta(kind):
    c = Cached(requests(kind, [60_000]), 8, 1, 128, 32, 12, uniform=True)
    c.check()
    assert not counters(c).any()


@pytest.mark.parametrize("kind", ["token", "draft"])
def test_a_long_request_whose_rows_see_nothing(kind):
    lim = requests(kind, [9000, 40])
    lim[1] = [0] * len(lim[1])
    c = Cached(lim, 64, 8, 64, 16, 13, uniform=True, extra=200)
    c.check()
    lim[0] = [0] * len(lim[0])
    Cached(lim, 64, 8, 64, 16, 13, uniform=True, extra=200).check()


@pytest.mark.parametrize("kind", ["token", "draft"])
def test_two_streams_with_a_workspace_each(kind):
    a, b = (Cached(requests(kind, [9000 + s]), 64, 8, 64, 16, 14 + s, uniform=True) for s in (0, 1))
    want = [x.run().clone() for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, s in zip((a, b), streams):
            x.run(stream=s)
    torch.cuda.synchronize()
    for x, w in zip((a, b), want):
        assert int(x.err.item()) == 0 and not counters(x).any()
        assert torch.equal(x.out.view(torch.int16), w.view(torch.int16))


@pytest.mark.parametrize("kind", ["token", "draft"])
@pytest.mark.parametrize("lengths", [[9000], [700] * 3])
def test_counters_that_were_not_zero_are_reported(kind, lengths):
    c = Cached(requests(kind, lengths), 64, 8, 64, 16, 15, uniform=True, extra=200)
    want = c.run().clone()
    c.ws[:4096].view(torch.int32).fill_(1000)  # more than parts can have arrived
    c.run()
    torch.cuda.synchronize()
    assert int(c.err.item()) == _native.ERR_WORKSPACE
    c.ws.zero_()
    c.err.zero_()
    c.out = torch.empty_like(want, dtype=BF)
    got = c.run()
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
