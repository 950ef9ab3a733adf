"""Ways of calling the attentions: as many requests as a call takes."""
import pytest
import torch

from test_gpu_attn import Cached, Prompt, draft

pytestmark = pytest.mark.gpu


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
