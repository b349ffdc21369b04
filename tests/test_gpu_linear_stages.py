"""Products of E4M3 blocks one after the other without a pause, with fewer, as many and more blocks
than the kernels have stages: every CTA leaves its shared memory as the next kernel expects it."""
import pytest
import torch

import layer_ref as ref
from attention_ref import check
from block_draft_proposal_gb300 import dflash2

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("rows", [[1, 16], [20, 64], [70, 300], [1, 50, 270]])
def test_back_to_back(cuda, rows):
    n_out, runs = 260, []
    for i, blocks in enumerate([1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 13, 16, 17]):
        n_in = 128 * blocks - 16 * (i % 8)
        x_q, x_s = ref.quantise_blocks(ref.rows(rows[i % len(rows)], n_in, BF, i).float())
        w_q, w_s = ref.weights(n_out, n_in, i + 1)
        runs.append((x_q, x_s, w_q, w_s, [t.cuda() for t in (x_q, w_q, w_s, x_s)]))
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    torch.cuda.synchronize()
    got = [[dflash2.linear_fp8_blocks(*run[4], err=err)[0] for run in runs] for _ in range(20)]
    torch.cuda.synchronize()
    assert int(err) == 0
    for i, (x_q, x_s, w_q, w_s, _) in enumerate(runs):
        want, bound = ref.product(x_q, x_s, w_q, w_s)
        check(f"run {i}", got[0][i], want, bound + ref.HALF_STEP[BF] * want.abs())
        assert all(torch.equal(again[i], got[0][i]) for again in got)
