"""Exponent bytes of an E4M3 cache outside [79, 175], which no write leaves: every path
takes the nearest byte of that range."""
import pytest
import torch

from attention_ref import e4m3_values
from block_draft_proposal_gb300 import dflash2
from test_gpu_attention import BF, F32, Case

pytestmark = pytest.mark.gpu
BYTES = (0, 1, 40, 78, 79, 127, 175, 176, 200, 254, 255)


def _pair(c):
    """The case's cache with odd exponent bytes, and with the nearest ones in range."""
    g = torch.Generator().manual_seed(3)
    odd = [torch.tensor(BYTES, dtype=torch.uint8)[torch.randint(0, len(BYTES), e.shape, generator=g)]
           for e in (c.cache.k_exp, c.cache.v_exp)]
    return (dflash2.KVCache(c.cache.k, c.cache.v, *(e.cuda() for e in odd)),
            dflash2.KVCache(c.cache.k, c.cache.v, *(e.clamp(79, 175).cuda() for e in odd)))


@pytest.mark.parametrize("t,hq,hk,d,ps,dtype", [
    ([1, 2], 4, 2, 128, 16, BF), ([2, 1], 4, 2, 64, 32, BF),      # few rows a request
    ([20, 40], 8, 2, 128, 16, BF), ([30, 20], 4, 1, 64, 64, BF),  # many
    ([3, 1], 4, 2, 128, 24, BF), ([3, 1], 4, 2, 64, 16, F32)])    # CUDA cores
def test_attention(cuda, t, hq, hk, d, ps, dtype):
    c = Case(t, [150, 40], hq, hk, d, ps, dtype=dtype, e4m3=True, seed=5)
    odd, near = _pair(c)
    args = (c.table.cuda(), c.cu.cuda(), c.lens.cuda(), 0.1)
    a, la, err = dflash2.tree_attention(c.q, odd, *args, with_lse=True)
    b, lb, _ = dflash2.tree_attention(c.q, near, *args, with_lse=True)
    assert int(err.item()) == 0
    assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.isnan(la), torch.isnan(lb))
    assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
    assert torch.equal(la.nan_to_num(7.0), lb.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,ps", [(64, 16), (128, 32), (256, 16), (80, 7)])
def test_read(cuda, d, ps, dtype):
    c = Case([3], [150], 2, 2, d, ps, e4m3=True, seed=6)
    odd, near = _pair(c)
    slots = c.slots.cuda()
    k, v, err = dflash2.kv_cache_read(odd, slots, dtype=dtype)
    assert int(err.item()) == 0
    page, off = c.slots // ps, c.slots % ps
    for got, codes, exps in ((k, near.k, near.k_exp), (v, near.v, near.v_exp)):
        scale = 2.0 ** (exps.cpu()[page, :, off].double() - 127)
        want = e4m3_values()[codes.cpu()[page, :, off].long()] * scale[..., None]
        assert torch.equal(got.cpu().double(), want)
