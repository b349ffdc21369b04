"""The product of E4M3 blocks on the GPU, against 64 bits."""
import math

import pytest
import torch

import layer_ref as ref
from attention_ref import check
from block_draft_proposal_gb300 import dflash2

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _check(y, x_q, x_s, w_q, w_s, name):
    want, bound = ref.product(x_q.cpu(), x_s.cpu(), w_q.cpu(), w_s.cpu())
    check(name, y, want, bound + ref.HALF_STEP[y.dtype] * want.abs())


SHAPES = [  # rows, in, out
    (1, 16, 1), (1, 128, 128), (1, 4096, 384), (3, 2560, 20000), (16, 2576, 7000), (9, 1040, 260), (2, 144, 130), (7, 1936, 1001), (16, 256, 257), (17, 384, 96),
    (33, 512, 640), (48, 1040, 200), (64, 128, 300), (65, 640, 128), (100, 2048, 130), (128, 256, 512),
    (129, 1296, 511), (200, 400, 264), (256, 256, 256), (257, 144, 1030), (300, 1152, 384), (513, 272, 520),
    (1000, 656, 776), (1500, 128, 144),
    # tiles of 64, 128 and 256 columns; more tiles than pairs of CTAs; the last ones ragged
    (70, 272, 6001), (256, 400, 6016), (300, 144, 5000), (300, 272, 5001), (1100, 272, 9003), (2500, 144, 2600)]


@pytest.mark.parametrize("rows,n_in,n_out", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_product(cuda, rows, n_in, n_out, dtype):
    x = ref.rows(rows, n_in, dtype, rows + n_in)
    w_q, w_s = ref.weights(n_out, n_in, 5)
    x_q, x_s = ref.quantise_blocks(x.float())
    name = f"{rows}x{n_in}x{n_out}"
    y, err = dflash2.linear_fp8_blocks(x.cuda(), w_q.cuda(), w_s.cuda())
    assert int(err) == 0 and y.dtype == dtype
    _check(y, x_q, x_s, w_q, w_s, name)
    # the codes and scales of the call are the quantisation's, and fp32 results their sums
    codes, scales = dflash2.quantize_blocks_e4m3(x.cuda())
    y2, err = dflash2.linear_fp8_blocks(codes, w_q.cuda(), w_s.cuda(), x_scale=scales, out_dtype=dtype)
    assert int(err) == 0 and torch.equal(y2, y)


@pytest.mark.parametrize("rows,n_out", [(1, 400), (5, 400), (40, 400), (130, 400), (700, 400), (90, 6008),
                                        (2600, 2500), (130, 399), (700, 401), (90, 6007), (2601, 2501)])
def test_whole_numbers_are_exact(cuda, rows, n_out):
    g = torch.Generator().manual_seed(rows)
    n_in = 656
    x = torch.randint(-8, 9, (rows, n_in), generator=g).float()
    w = torch.randint(-8, 9, (n_out, n_in), generator=g).float()
    x_s = 2.0 ** torch.randint(-3, 4, (rows, 6), generator=g).float()
    w_s = 2.0 ** torch.randint(-3, 4, (-(-n_out // 128), 6), generator=g).float()
    code = ref.encode(x.double()), ref.encode(w.double())
    y, _ = dflash2.linear_fp8_blocks(code[0].cuda(), code[1].cuda(), w_s.cuda(), x_scale=x_s.cuda(), out_dtype=F32)
    want, _ = ref.product(code[0], x_s, code[1], w_s)
    assert torch.equal(y.cpu().double(), want)


@pytest.mark.parametrize("rows", [3, 90, 600])
def test_nan_stays_in_its_row_and_column(cuda, rows):
    n_in, n_out = 272, 300
    x_q, x_s = ref.quantise_blocks(ref.rows(rows, n_in, F32, 1))
    w_q, w_s = ref.weights(n_out, n_in, 2)
    x_q[1, 200], w_q[7, 3] = 127, 255
    y, err = dflash2.linear_fp8_blocks(x_q.cuda(), w_q.cuda(), w_s.cuda(), x_scale=x_s.cuda(), out_dtype=F32)
    bad = torch.zeros((rows, n_out), dtype=torch.bool)
    bad[1], bad[:, 7] = True, True
    assert int(err) == 0 and torch.equal(torch.isnan(y).cpu(), bad)
    x = ref.rows(rows, n_in, F32, 1)
    x[2, 0] = math.inf                                         # no code: seen, not saturated
    y, _ = dflash2.linear_fp8_blocks(x.cuda(), w_q.cuda(), w_s.cuda())
    assert torch.isnan(y[2]).all() and not torch.isnan(y[0, 8:]).any()


@pytest.mark.parametrize("rows,dtype", [(50, BF), (11, BF), (16, F32), (1, BF)])
def test_strided_rows_and_zero_rows(cuda, rows, dtype):
    wide = ref.rows(rows, 700, dtype, 3).cuda()
    w_q, w_s = (t.cuda() for t in ref.weights(200, 320, 4))
    for at in (0, 8, 3):                                       # 3: off 16-byte alignment
        x = wide[:, at:at + 320]
        y, _ = dflash2.linear_fp8_blocks(x, w_q, w_s)
        want, _ = dflash2.linear_fp8_blocks(x.contiguous(), w_q, w_s)
        assert torch.equal(y, want)
    wide[rows // 7, :320] = 0
    y, _ = dflash2.linear_fp8_blocks(wide[:, :320], w_q, w_s)
    assert not y[rows // 7].any()
    y, _ = dflash2.linear_fp8_blocks(wide[:0, :320], w_q, w_s)
    assert y.shape == (0, 200)


@pytest.mark.parametrize("rows", [2, 60, 300])
def test_what_lies_behind_the_result_stays(cuda, rows):
    """Outputs end inside a buffer; its neighbours keep their values."""
    n_in, n_out = 384, 321
    x = ref.rows(rows, n_in, BF, 6).cuda()
    w_q, w_s = (t.cuda() for t in ref.weights(n_out, n_in, 7))
    flat = torch.full((rows * n_out + 4096,), 7.0, dtype=BF, device=cuda)
    out = flat[1024:1024 + rows * n_out].view(rows, n_out)
    dflash2.linear_fp8_blocks(x, w_q, w_s, out=out)
    want, _ = dflash2.linear_fp8_blocks(x, w_q, w_s)
    assert torch.equal(out, want) and bool((flat[:1024] == 7).all()) and bool((flat[1024 + rows * n_out:] == 7).all())


def test_rows_do_not_depend_on_their_neighbours(cuda):
    """Calls of one kernel agree bit for bit row by row, and twice."""
    x = ref.rows(500, 512, BF, 8).cuda()
    w_q, w_s = (t.cuda() for t in ref.weights(300, 512, 9))
    y, _ = dflash2.linear_fp8_blocks(x, w_q, w_s)
    again, _ = dflash2.linear_fp8_blocks(x, w_q, w_s)
    moved, _ = dflash2.linear_fp8_blocks(x.flip(0), w_q, w_s)
    assert torch.equal(y, again) and torch.equal(moved.flip(0), y)


@pytest.mark.parametrize("rows", [3, 400])
def test_streams_and_graphs(cuda, rows):
    x = ref.rows(rows, 1024, BF, 10).cuda()
    w_q, w_s = (t.cuda() for t in ref.weights(260, 1024, 11))
    want, _ = dflash2.linear_fp8_blocks(x, w_q, w_s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, err = dflash2.linear_fp8_blocks(x, w_q, w_s, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and int(err) == 0
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    ws = torch.empty(dflash2.linear_fp8_blocks_workspace_size(rows, 1024, 260), dtype=torch.uint8, device=cuda)
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    with torch.cuda.graph(graph):
        dflash2.linear_fp8_blocks(x, w_q, w_s, out=out, workspace=ws, err=err)
    x.copy_(x.flip(0))
    for _ in range(2):
        graph.replay()
    assert torch.equal(out.flip(0), want) and int(err) == 0
