"""Many query heads per key/value head (up to 128): a token's rows fill more than one
block of rows, and blocks begin inside a token."""
import pytest

from block_draft_proposal_gb300 import dflash2
from test_gpu_attention import BF, Case, _check_prompt, _prompt

pytestmark = pytest.mark.gpu
GROUPS = [(65, 1, 64), (71, 1, 64), (80, 1, 128), (96, 1, 128), (128, 1, 64), (192, 2, 128), (127, 1, 128)]


@pytest.mark.parametrize("words", [None, 1], ids=["chain", "tree"])
@pytest.mark.parametrize("hq,hk,d", GROUPS)
def test_over_an_e4m3_cache_with_empty_requests(cuda, hq, hk, d, words):
    """Few rows a request on average, because most requests are empty."""
    t = [1, 0, 2, 0, 0, 3, 0, 0] + [0] * 8
    ctx = [300, 9, 5, 0, 0, 1500, 1, 128] + [0] * 8
    assert sum(t) * (hq // hk) <= 48 * len(t)
    c = Case(t, ctx, hq, hk, d, 16, e4m3=True, words=words, seed=hq, empty_row=1 if words else None)
    out, lse, err = c.run()
    assert int(err.item()) == 0
    c.check(out, lse)


@pytest.mark.parametrize("e4m3", [False, True], ids=["native", "e4m3"])
@pytest.mark.parametrize("hq,hk,d", GROUPS)
def test_with_a_token_or_more_in_every_request(cuda, hq, hk, d, e4m3):
    c = Case([1, 3, 1], [200, 70, 0], hq, hk, d, 32, e4m3=e4m3, words=1, seed=hq + 1)
    out, lse, err = c.run()
    assert int(err.item()) == 0
    c.check(out, lse)


@pytest.mark.parametrize("hq,hk,d", GROUPS)
def test_prompts(cuda, hq, hk, d):
    lens = [5, 131, 1]
    qkv_dev, qkv, cu = _prompt(lens, hq, hk, d, BF, 700 + hq)
    out, lse, err = dflash2.prompt_attention(*qkv_dev, cu.cuda(), d ** -0.5, with_lse=True)
    assert int(err.item()) == 0
    _check_prompt(lens, hq, hk, qkv, out, lse, d ** -0.5, BF)
