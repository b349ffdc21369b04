"""Attention over an E4M3 cache whose value scales lie far apart."""
import pytest
import torch

from test_gpu_attention import BF, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [16, 40], ids=["64rows", "160rows"])
@pytest.mark.parametrize("loud,main", [(3, 5), (3, 2999), (2999, 5), (2000, 2001)])
@pytest.mark.parametrize("span", [7, 8, 9, 12, 16, 20, 22, 23])
def test_a_loud_value_of_a_key_that_hardly_counts(cuda, span, loud, main, t):
    """One key takes half of the weight and thousands of small ones, of one sign, the other half;
    a key of next to no weight has a value row 2^span above theirs."""
    ctx = 3000
    c = Case([t], [ctx], 4, 1, 64, 64, e4m3=True, seed=17)
    q = torch.zeros(t, 4, 64)
    q[..., 0] = 1.0
    c.q_host = q.to(BF)
    c.q = c.q_host.cuda()
    c.scale = 1.0
    c.k_rows.fill_(0.0)
    c.k_rows[main, :, 0] = 8.0           # the other keys' weights are e^-8 of this one's
    c.k_rows[loud, :, 0] = -20.0
    c.v_rows.copy_(c.v_rows.abs().clamp(1.0, 1.75))
    c.v_rows[loud] *= 2.0 ** span
    c.write()
    out, lse, err = c.run()
    assert int(err.item()) == 0
    c.check(out, lse)
