"""The E4M3 cache's attention where requests have few rows, at the places where the
kernel's own rules turn: several row blocks in a ragged batch, the average that
selects it, weights far below a row's largest, uneven splits."""
import pytest
import torch

from test_gpu_attention import BF, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("words", [None, 2], ids=["chain", "tree"])
@pytest.mark.parametrize("hq,hk,d,ps", [(8, 2, 128, 16), (8, 1, 64, 32), (5, 1, 128, 128),
                                        (6, 2, 64, 256)])
def test_a_ragged_batch_with_long_requests(cuda, hq, hk, d, ps, words):
    """Few rows on average; one request has several blocks of them, one none."""
    t = [1] * 20 + [100, 0, 37, 2]
    ctx = [(97 * i * i) % 700 for i in range(20)] + [129, 300, 0, 1500]
    c = Case(t, ctx, hq, hk, d, ps, e4m3=True, words=words, seed=11)
    out, lse, err = c.run()
    assert int(err.item()) == 0
    c.check(out, lse)


@pytest.mark.parametrize("last", [12, 13])
def test_both_sides_of_the_average(cuda, last):
    c = Case([12, 12, 12, last], [700, 127, 128, 1900], 8, 2, 128, 16, e4m3=True, words=1, seed=12)
    out, lse, err = c.run()
    assert int(err.item()) == 0
    c.check(out, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gap", [6.0, 14.0, 15.5, 40.0])
@pytest.mark.parametrize("at", [3, 2999])
def test_one_key_far_above_the_rest(cuda, gap, at, d):
    """Thousands of small weights of one sign beside one large, early and late."""
    c = Case([1, 2], [6000, 3000], 4, 1, d, 64, e4m3=True, seed=13)
    q = torch.zeros(3, 4, d)
    q[..., 0] = 1.0
    c.q_host = q.to(BF)
    c.q = c.q_host.cuda()
    c.scale = 1.0
    c.k_rows.fill_(0.0)
    c.k_rows[at, :, 0] = gap
    c.k_rows[6001 + min(at, 2000), :, 0] = gap
    c.v_rows.copy_(c.v_rows.abs().clamp(0.25, 4.0))
    c.write()
    out, lse, err = c.run()
    assert int(err.item()) == 0
    c.check(out, lse)


@pytest.mark.parametrize("tree", [False, True])
def test_an_uneven_batch(cuda, tree):
    g = torch.Generator().manual_seed(14)
    t = torch.randint(0, 14, (200,), generator=g).tolist()
    ctx = torch.randint(0, 900, (200,), generator=g).tolist()
    c = Case(t, ctx, 10, 2, 128, 16, e4m3=True, words=1 if tree else None, seed=15, empty_row=3)
    out, lse, err = c.run()
    assert int(err.item()) == 0
    c.check(out, lse, only=set(range(0, 200, 9)))
    again, lse2, _ = c.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
