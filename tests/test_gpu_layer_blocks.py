"""E4M3 blocks that the norms write, their scales by their own values; and products of up to 64 rows
whose blocks are split over every number of CTAs, against 64 bits."""
import pytest
import torch

import layer_ref as ref
from attention_ref import U_F32, check
from block_draft_proposal_gb300 import dflash2

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
WIDTHS = [1, 7, 128, 130, 640, 1000, 1024, 1032, 4096, 4097, 7168, 8200, 9999, 16384, 20001, 32768]


def _weight(n, dtype, seed):
    return (1 + 0.3 * torch.randn(n, generator=torch.Generator().manual_seed(seed))).to(dtype)


def _blockwise_max(t):
    n, cols = t.shape
    blocks = -(-cols // 128)
    return torch.nn.functional.pad(t.abs(), (0, blocks * 128 - cols)).view(n, blocks, 128).amax(-1)


def _check_scales(scale, want, bound):
    """A block's scale is its largest magnitude / 448, that magnitude off by what the values may be off, the
    division rounded (half a step); 1 where all are zeros."""
    top, off = _blockwise_max(want), _blockwise_max(bound)
    allowed = off / 448 + 2 * U_F32 * top / 448
    expected = torch.where(top > 0, top / 448, torch.ones_like(top))
    over = ((scale.cpu().double() - expected).abs() - allowed).max()
    assert float(over) <= 0, f"a scale is off by {float(over)} more than its values"


@pytest.mark.parametrize("hidden", WIDTHS)
@pytest.mark.parametrize("xt,wt", [(BF, BF), (F32, BF), (F32, F32), (BF, F32)])
def test_scales_of_a_norm(cuda, hidden, xt, wt):
    x, w = ref.rows(3, hidden, xt, 1), _weight(hidden, wt, 2)
    x[1, :min(hidden, 128)] = 0                                # a block of zeros
    codes, scale = dflash2.sublayer_norm(x.cuda(), w.cuda(), eps=1e-5, e4m3=True)
    want, _ = ref.norm(x.double(), w.double(), 0.0, 1e-5)
    bound = ref.NORM * want.abs()
    _check_scales(scale, want, bound)
    ref.held_as_blocks(codes, scale, want, bound + ref.TINY, "norm")


@pytest.mark.parametrize("hidden", WIDTHS)
@pytest.mark.parametrize("rt,dt", [(BF, BF), (F32, BF), (F32, F32), (BF, F32)])
def test_scales_of_a_join(cuda, hidden, rt, dt):
    res, y, gate = ref.rows(3, hidden, rt, 3), ref.rows(3, hidden, dt, 4), ref.rows(3, hidden, dt, 5)
    wp, wn = _weight(hidden, dt, 6), _weight(hidden, dt, 7)
    dev = [t.cuda() for t in (res, y, wp, gate, wn)]
    _, codes, scale = dflash2.sublayer_join(dev[0], dev[1], post_weight=dev[2], gate=dev[3], gate_act="tanh",
                                            branch_scale=0.5, next_weight=dev[4], e4m3=True)
    _, _, want, off = ref.join(res.double(), y.double(), wp.double(), gate.double(), "tanh", 0.5, wn.double(), 0.0, 1e-6)
    _check_scales(scale, want, off)
    ref.held_as_blocks(codes, scale, want, off + ref.TINY, "join")


@pytest.mark.parametrize("hidden", [8, 128, 136, 1000, 1024, 1032, 4096, 7168, 8200, 16384, 32768])
@pytest.mark.parametrize("xt", [BF, F32])
def test_blocks_are_those_of_the_values(cuda, hidden, xt):
    """Rows of whole 16-byte pieces are summed the same way whatever is written, so that the codes and scales
    are bit for bit the quantisation of the fp32 result."""
    x, y, w = ref.rows(5, hidden, xt, 8).cuda(), ref.rows(5, hidden, F32, 9).cuda(), _weight(hidden, F32, 10).cuda()
    plain, _ = dflash2.sublayer_norm(x, w, eps=1e-5)
    codes, scale = dflash2.sublayer_norm(x, w, eps=1e-5, e4m3=True)
    want_c, want_s = ref.quantise_blocks(plain.cpu())
    assert torch.equal(scale.cpu(), want_s) and ref.same_codes(codes, want_c)
    args = dict(post_weight=w, next_weight=w, gate=y, gate_act="sigmoid")
    r, plain, _ = dflash2.sublayer_join(x, y, **args)
    r2, codes, scale = dflash2.sublayer_join(x, y, e4m3=True, **args)
    want_c, want_s = ref.quantise_blocks(plain.cpu())
    assert torch.equal(r, r2) and torch.equal(scale.cpu(), want_s) and ref.same_codes(codes, want_c)


# Blocks go over 8, 5, 4 or 2 CTAs, by the tiles of 128 outputs (304 CTAs at most) and the blocks (two each):
# splits that leave CTAs uneven runs of blocks, and 5 uneven shares of the rows
@pytest.mark.parametrize("rows", [17, 32, 33, 50, 64])
@pytest.mark.parametrize("n_in,n_out", [(2048, 260), (2416, 400), (4752, 129), (1296, 5000), (1664, 5001), (2672, 7600),
                                        (1040, 9700),
                                        (1040, 300), (1536, 9000), (528, 300), (656, 19000)])
def test_few_rows_split(cuda, rows, n_in, n_out):
    x = ref.rows(rows, n_in, BF, rows + n_in)
    w_q, w_s = ref.weights(n_out, n_in, n_out)
    x_q, x_s = ref.quantise_blocks(x.float())
    want, bound = ref.product(x_q, x_s, w_q, w_s)
    w_q, w_s = w_q.cuda(), w_s.cuda()
    y, err = dflash2.linear_fp8_blocks(x_q.cuda(), w_q, w_s, x_scale=x_s.cuda(), out_dtype=F32)
    assert int(err) == 0
    check("fp32", y, want, bound + ref.HALF_STEP[F32] * want.abs())
    y, err = dflash2.linear_fp8_blocks(x.cuda(), w_q, w_s)
    assert int(err) == 0
    check("bf16", y, want, bound + ref.HALF_STEP[BF] * want.abs())


@pytest.mark.parametrize("n_in,n_out", [(2416, 400), (1664, 5001), (272, 130)])
def test_results_by_the_number_of_rows(cuda, n_in, n_out):
    """A row's result is the same among up to 64 rows, and among more."""
    x = ref.rows(1100, n_in, BF, 11).cuda()
    w_q, w_s = (t.cuda() for t in ref.weights(n_out, n_in, 12))

    def run(rows):
        return dflash2.linear_fp8_blocks(x[:rows], w_q, w_s, out_dtype=F32)[0]

    few, many = run(64), run(1100)
    for rows in (1, 2, 5, 16, 17, 32, 33):
        assert torch.equal(run(rows), few[:rows])
    for rows in (65, 200, 300, 700):
        assert torch.equal(run(rows), many[:rows])
