"""Values that are not finite where each CTA takes many short pieces of work one after
the other: every row that sees one shows it, and no other row does."""
import math

import pytest
import torch

from block_draft_proposal_gb300 import dflash2
from test_gpu_attention import BF, NAN, Case, _check_prompt, _prompt

pytestmark = pytest.mark.gpu


def _spoil(c, every, bads):
    """A drafted value row of every `every`-th request is not finite, in all heads."""
    at, n = 0, 0
    for b, (t, ctx) in enumerate(zip(c.t, c.ctx)):
        if t and b % every == 0:
            c.v_rows[at + ctx + (b // every) % t] = bads[n % len(bads)]
            n += 1
        at += t + ctx
    c.write()


def _run(c):
    """The same three times: what a row shows does not depend on when pieces are taken."""
    out, lse, err = c.run()
    assert int(err.item()) == 0
    c.check(out, lse)
    for _ in range(2):
        again, lse2, _ = c.run()
        assert torch.equal(torch.isnan(again), torch.isnan(out)) and torch.equal(lse, lse2)
        assert torch.equal(again.nan_to_num(0.0, 1.0, -1.0), out.nan_to_num(0.0, 1.0, -1.0))


@pytest.mark.parametrize("words", [None, 1], ids=["chain", "tree"])
@pytest.mark.parametrize("every", [1, 2, 5])
@pytest.mark.parametrize("d", [64, 128])
def test_short_requests_over_a_native_cache(cuda, d, every, words):
    t = [1 + i % 3 for i in range(64)]
    ctx = [(i * 31) % 100 for i in range(64)]
    c = Case(t, ctx, 16, 8, d, 16, words=words, seed=every)
    _spoil(c, every, (NAN, math.inf, -math.inf))
    _run(c)


@pytest.mark.parametrize("words", [None, 1], ids=["chain", "tree"])
@pytest.mark.parametrize("every", [1, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_short_requests_with_many_rows_over_an_e4m3_cache(cuda, d, every, words):
    t = [13 + i % 4 for i in range(64)]                  # 52 to 64 rows
    ctx = [(i * 31) % 100 for i in range(64)]
    c = Case(t, ctx, 32, 8, d, 16, e4m3=True, words=words, seed=every)
    _spoil(c, every, (NAN,))
    _run(c)


@pytest.mark.parametrize("d", [64, 128])
def test_short_requests_with_few_rows_over_an_e4m3_cache(cuda, d):
    c = Case([1 + i % 3 for i in range(64)], [(i * 31) % 100 for i in range(64)], 16, 8, d, 16, e4m3=True,
             words=1, seed=9)
    _spoil(c, 1, (NAN,))
    _run(c)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("each", [1, 2])
def test_short_prompts(cuda, each, d):
    lens = [1 + (i * 13) % 60 for i in range(200)]
    hq, hk = 8, 4
    (q, k, v), qkv, cu = _prompt(lens, hq, hk, d, BF, 800 + each)
    at = 0
    for b, n in enumerate(lens):
        if b % each == 0:
            bad = (NAN, math.inf, -math.inf)[b % 3]
            qkv[at + (b * 7) % n, hq + hk:hq + 2 * hk] = bad
        at += n
    dev = qkv.cuda()
    rows = dev[:, :hq], dev[:, hq:hq + hk], dev[:, hq + hk:hq + 2 * hk]
    for _ in range(3):
        out, lse, err = dflash2.prompt_attention(*rows, cu.cuda(), d ** -0.5, with_lse=True)
        assert int(err.item()) == 0
        _check_prompt(lens, hq, hk, qkv, out, lse, d ** -0.5, BF)


@pytest.mark.parametrize("e4m3", [False, True], ids=["native", "e4m3"])
@pytest.mark.parametrize("t,hq", [(33, 4), (40, 4), (64, 4), (43, 5)])      # 132 to 256 rows
@pytest.mark.parametrize("d", [64, 128])
def test_row_blocks_that_fill_both_slots(cuda, d, t, hq, e4m3):
    """A warp writes whole output rows, and each row's own thread adds the values that
    are not finite."""
    c = Case([t] * 40, [(i * 31) % 60 for i in range(40)], 2 * hq, 2, d, 16, e4m3=e4m3, words=1, seed=t)
    _spoil(c, 1, (NAN,) if e4m3 else (NAN, math.inf, -math.inf))
    _run(c)


@pytest.mark.parametrize("d", [64, 128])
def test_longer_prompts(cuda, d):
    lens, hq, hk = [200, 333, 129, 257, 70, 65], 8, 2
    _, qkv, cu = _prompt(lens, hq, hk, d, BF, 880)
    at = 0
    for b, n in enumerate(lens):
        for i, bad in ((n // 3, NAN), (n // 2, math.inf), (n - 1, -math.inf)):
            qkv[at + i, hq + hk:, (b + i) % d] = bad
        at += n
    dev = qkv.cuda()
    out, lse, err = dflash2.prompt_attention(dev[:, :hq], dev[:, hq:hq + hk], dev[:, hq + hk:], cu.cuda(),
                                             d ** -0.5, with_lse=True)
    assert int(err.item()) == 0
    _check_prompt(lens, hq, hk, qkv, out, lse, d ** -0.5, BF)
