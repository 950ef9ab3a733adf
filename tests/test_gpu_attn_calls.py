"""Ways of calling the attentions: captured in a graph where every CTA runs at
once, with as many requests as a call takes, and with the output in the queries."""
import pytest
import torch

from test_gpu_attn import Cached, Prompt, draft

pytestmark = pytest.mark.gpu


def requests(kind, lengths):
    return [[n] if kind == "token" else draft(n, n % 8) for n in lengths]


def bits(x):
    return x.view(torch.int16)


@pytest.mark.parametrize("kind", ["token", "draft"])
@pytest.mark.parametrize("Hq, Hkv, D", [(64, 8, 64), (8, 1, 128), (32, 4, 128)])
@pytest.mark.parametrize("lengths", [[9000], [2300, 1], [9000, 60, 5001]])
def test_graphs_of_long_requests(kind, Hq, Hkv, D, lengths):
    """Tables of 2048 keys and more with few requests: parts are added up by all CTAs
    (cooperative launch).  Replays with changed inputs, eager calls between them."""
    a, b = (Cached(requests(kind, lengths), Hq, Hkv, D, 16, 20 + s, uniform=True, extra=200) for s in (0, 1))
    a.check()
    wants = [x.run().clone() for x in (a, b)]
    inputs = [[t.clone() for t in (x.q, x.cache, x.table)] for x in (a, b)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    for i in range(6):
        for dst, src in zip((a.q, a.cache, a.table), inputs[i % 2]):
            dst.copy_(src)
        a.out.fill_(float("nan"))
        graph.replay()
        if i % 3 == 2:  # the same workspace, right after
            again = a.run(out=torch.empty_like(a.out))
            assert torch.equal(bits(again), bits(wants[i % 2]))
        torch.cuda.synchronize()
        assert torch.equal(bits(a.out), bits(wants[i % 2]))
        assert int(a.err.item()) == 0 and not a.ws[:4096].any()


MOST = 2048  # PE_MAX_ATTN_B


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["token", "wide token", "draft"])
@pytest.mark.parametrize("uniform", [True, False])
def test_the_largest_number_of_requests(kind, D, uniform):
    g = torch.Generator().manual_seed(21)
    n = torch.randint(1, 80, (MOST,), generator=g).tolist()
    n[700], n[2047] = 3000, 900
    lim = [draft(x, x % 8) if kind == "draft" and b % 7 == 0 or kind == "draft" and uniform else [x] for b, x in enumerate(n)]
    if not uniform:
        lim[5] = lim[1500] = []
    Cached(lim, 12 if kind == "wide token" else 4, 1, D, 16, 22, uniform=uniform).check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("uniform", [True, False])
def test_the_largest_number_of_prompts(D, uniform):
    g = torch.Generator().manual_seed(23)
    lens = [9] * MOST if uniform else torch.randint(0, 40, (MOST,), generator=g).tolist()
    if not uniform:
        lens[1000] = 1200
    Prompt(lens, 4, 1, D, 24, uniform=uniform).check()


@pytest.mark.parametrize("kind", ["token", "draft", "prompt"])
@pytest.mark.parametrize("lengths", [[9000], [700, 33, 150] * 20])
def test_output_in_the_queries(kind, lengths):
    """out may be q: a row's query is read before its result is written, and by no other row."""
    if kind == "prompt":
        c = Prompt(lengths, 16, 2, 64, 25, fused=False)
        c.q = c.q.contiguous()
    else:
        c = Cached(requests(kind, lengths), 16, 2, 64, 16, 25, uniform=True, extra=200)
    want, q = c.run().clone(), c.q.clone()
    for _ in range(5):
        c.q.copy_(q)
        c.run(out=c.q)
        torch.cuda.synchronize()
        assert int(c.err.item()) == 0 and torch.equal(bits(c.q), bits(want))
