"""Prompts with values that are not finite between many that are shorter than
one stream's rows."""
import pytest
import torch

from test_gpu_attn import Prompt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D, Hq, Hkv", [(64, 16, 2), (128, 8, 1)])
@pytest.mark.parametrize("shorts", [7, 8, 20])
@pytest.mark.parametrize("n", [40, 200])
def test_infinities_between_short_prompts(D, Hq, Hkv, shorts, n):
    """Each long prompt holds infinities in places that its first rows do not see;
    the rows that do see them get them, and no other prompt does."""
    lens = ([n] + [1 + i % 16 for i in range(shorts)]) * (1600 // (shorts + 1))
    want = Prompt(lens, Hq, Hkv, D, 8).run().clone()
    p = Prompt(lens, Hq, Hkv, D, 8)
    expected, at, k = want.clone(), 0, 0
    for length in lens:
        if length == n:
            t, h, d = at + n // 2 + k % (n // 2), k % Hkv, (7 * k) % D
            what = float("inf") if k % 3 else float("nan")
            p.v[t, h, d] = what
            expected[t:at + n, h * Hq // Hkv:(h + 1) * Hq // Hkv, d] = what
            k += 1
        at += length
    for _ in range(3):
        got = p.run(out=torch.empty_like(want))
        torch.cuda.synchronize()
        assert int(p.err.item()) == 0
        assert torch.equal(got.isnan(), expected.isnan())
        assert torch.equal(got.nan_to_num(0.0, 3e38, -3e38), expected.nan_to_num(0.0, 3e38, -3e38))
