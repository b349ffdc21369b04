"""Packed prompts whose cu_q falls: the clamped requests overlap and may hold more rows
than there are tokens, and every token that one of them holds is written."""
import math

import pytest
import torch

import attention_ref as ref
from block_draft_proposal_gb300 import dflash2
from test_gpu_attention import BF, F32, _out_u, _prompt, _weights_u

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [(F32, 64), (F32, 128), (BF, 80), (BF, 64), (BF, 128)])
@pytest.mark.parametrize("cu,first", [([0, 900, 100, 1000], 100), ([0, 600, 0, 600, 0, 600, 0, 1000], 0)])
def test_tokens_of_the_last_request(cuda, cu, first, dtype, d):
    n = 1000
    (q, k, v), qkv, _ = _prompt([n], 2, 1, d, dtype, 900)
    out = torch.full((n, 2, d), math.nan, dtype=dtype, device=cuda)
    _, _, err = dflash2.prompt_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device=cuda),
                                         d ** -0.5, out=out)
    assert int(err.item()) == dflash2.DEVERR_ID_RANGE
    assert torch.isfinite(out).all()
    x = qkv[first:].double()
    want, _, bound, _ = ref.attend(x[:, :2], x[:, 2:3], x[:, 3:4], ref.chain_or_tree(n - first, 0, None),
                                   d ** -0.5, _weights_u(dtype, False), _out_u(dtype))
    ref.check("tokens in the last request alone", out[900:], want[900 - first:], bound[900 - first:])


@pytest.mark.parametrize("dtype,d", [(F32, 64), (BF, 64)])
def test_a_fall_behind_many_requests(cuda, dtype, d):
    """Behind some 300 requests of one token (more than a CTA looks at in one step)."""
    n, ones = 1000, 299
    (q, k, v), qkv, _ = _prompt([n], 2, 1, d, dtype, 901)
    cu = list(range(ones + 1)) + [900, 300, n]
    out = torch.full((n, 2, d), math.nan, dtype=dtype, device=cuda)
    _, _, err = dflash2.prompt_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device=cuda),
                                         d ** -0.5, out=out)
    assert int(err.item()) == dflash2.DEVERR_ID_RANGE
    assert torch.isfinite(out).all()
    own = torch.cat([qkv[:ones, 3:4]] * 2, 1).double()       # a token alone gets its own value
    assert float((out[:ones].double().cpu() - own).abs().max()) <= 1e-6
    x = qkv[300:].double()
    want, _, bound, _ = ref.attend(x[:, :2], x[:, 2:3], x[:, 3:4], ref.chain_or_tree(n - 300, 0, None),
                                   d ** -0.5, _weights_u(dtype, False), _out_u(dtype))
    ref.check("tokens in the last request alone", out[900:], want[600:], bound[600:])
