"""The norms around a sublayer and the E4M3 block quantisation on the GPU, against 64 bits."""
import math

import pytest
import torch

import layer_ref as ref
from attention_ref import check
from block_draft_proposal_gb300 import dflash2

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SHAPES = [(1, 1), (3, 7), (5, 64), (2, 1000), (9, 1024), (4, 1032), (33, 4096), (2, 7168), (3, 8200),
          (2, 9999), (3, 16384), (2, 20001), (1, 32768)]


def _weight(n, dtype, seed):
    return (1 + 0.3 * torch.randn(n, generator=torch.Generator().manual_seed(seed))).to(dtype)


@pytest.mark.parametrize("n,hidden", SHAPES)
@pytest.mark.parametrize("xt,wt", [(BF, BF), (F32, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_norm(cuda, n, hidden, xt, wt, e4m3):
    x, w = ref.rows(n, hidden, xt, 1), _weight(hidden, wt, 2)
    for offset in (0.0, 1.0):
        out, scale = dflash2.sublayer_norm(x.cuda(), w.cuda(), eps=1e-5, weight_offset=offset, e4m3=e4m3)
        want, _ = ref.norm(x.double(), w.double(), offset, 1e-5)
        bound = ref.NORM * want.abs() + ref.TINY
        if e4m3:
            ref.held_as_blocks(out, scale, want, bound, f"norm {n}x{hidden}")
        else:
            assert scale is None and out.dtype == wt
            check(f"norm {n}x{hidden}", out, want, bound + ref.HALF_STEP[wt] * want.abs())


@pytest.mark.parametrize("n,hidden", [(1, 5), (4, 256), (7, 1000), (3, 4096), (2, 8200), (2, 16392),
                                      (19, 511), (9, 513), (3, 4097), (5, 5001), (2, 16383), (2, 16385)])
@pytest.mark.parametrize("rt,dt", [(BF, BF), (F32, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("gate,act", [("none", "none"), ("channel", "tanh"), ("token", "sigmoid"),
                                      ("full", "sigmoid"), ("full", "none")])
@pytest.mark.parametrize("post,nxt", [(True, "native"), (False, "e4m3"), (True, "none")])
def test_join(cuda, n, hidden, rt, dt, gate, act, post, nxt):
    g = torch.Generator().manual_seed(hidden)
    res, y = ref.rows(n, hidden, rt, 3), ref.rows(n, hidden, dt, 4)
    wp, wn = _weight(hidden, dt, 5) if post else None, _weight(hidden, dt, 6) if nxt != "none" else None
    shape = {"none": None, "channel": (hidden,), "token": (n, 1), "full": (n, hidden)}[gate]
    gv = None if shape is None else (3 * torch.randn(shape, generator=g)).to(dt)
    dev = [None if t is None else t.cuda() for t in (res, y, wp, gv, wn)]
    r, out, scale = dflash2.sublayer_join(dev[0], dev[1], post_weight=dev[2], gate=dev[3], gate_act=act,
                                          branch_scale=-0.7, next_weight=dev[4], eps=1e-6, e4m3=nxt == "e4m3")
    wide = [None if t is None else t.double() for t in (res, y, wp, gv, wn)]
    branch = float(torch.tensor(-0.7, dtype=F32))
    want_r, dr, want, dout = ref.join(wide[0], wide[1], wide[2], wide[3], act, branch, wide[4], 0.0, 1e-6)
    check("residual", r, want_r, dr + ref.HALF_STEP[rt] * want_r.abs())
    assert torch.equal(dev[0].cpu(), res)                       # the residual itself stays
    if nxt == "none":
        assert out is None and scale is None
    elif nxt == "e4m3":
        ref.held_as_blocks(out, scale, want, dout + ref.TINY, "next norm")
    else:
        check("next norm", out, want, dout + ref.HALF_STEP[dt] * want.abs() + ref.TINY)


def test_rows_in_place_and_strided(cuda):
    n, hidden = 13, 520
    wide = ref.rows(n, 3 * hidden + 8, BF, 7).cuda()
    res, y, gate = wide[:, :hidden], wide[:, hidden:2 * hidden], wide[:, 2 * hidden:3 * hidden]
    w = _weight(hidden, BF, 8).cuda()
    args = dict(post_weight=w, gate_act="sigmoid", next_weight=w)
    r0, n0, _ = dflash2.sublayer_join(res.contiguous(), y.contiguous(), gate=gate.contiguous(), **args)
    before = wide.clone()
    r1, n1, _ = dflash2.sublayer_join(res, y, gate=gate, residual_out=res, **args)
    torch.cuda.synchronize()
    assert r1.data_ptr() == wide.data_ptr() and torch.equal(r1, r0) and torch.equal(n1, n0)
    assert torch.equal(wide[:, hidden:], before[:, hidden:])    # what lies between the rows stays
    # rows off 16-byte alignment take the same values by another path
    odd = wide[:, 1:hidden + 1]
    out, _ = dflash2.sublayer_norm(odd, w)
    want, _ = dflash2.sublayer_norm(odd.contiguous(), w)
    assert float((out.double() - want.double()).abs().max()) <= 2 * ref.HALF_STEP[BF] * float(want.abs().max())


def test_special_rows(cuda):
    hidden = 640
    x = ref.rows(6, hidden, F32, 9)
    x[0] = 0
    x[1, 5] = math.inf
    x[2, 130] = math.nan
    x[3] *= 1e-30
    x[4] *= 1e15
    w = _weight(hidden, F32, 10)
    out, _ = dflash2.sublayer_norm(x.cuda(), w.cuda(), eps=1e-6)
    out = out.cpu()
    assert torch.equal(out[0], torch.zeros(hidden))
    assert torch.isnan(out[2]).all() and torch.isnan(out[1, 5]) and not out[1, :5].any()
    want, _ = ref.norm(x[3:].double(), w.double(), 0.0, 1e-6)
    check("rows", out[3:], want, ref.NORM * want.abs() + ref.TINY)
    zero, _ = dflash2.sublayer_norm(x[:1].cuda(), w.cuda(), eps=0.0)
    assert torch.isnan(zero).all()
    codes, scale = dflash2.sublayer_norm(x.cuda(), w.cuda(), eps=1e-6, e4m3=True)
    assert not (codes[0] & 127).any() and torch.equal(scale[0].cpu(), torch.ones(5))
    assert ((codes[2] & 127) == 127).all()


def test_rows_do_not_depend_on_their_neighbours(cuda):
    x, w = ref.rows(301, 2048, BF, 11).cuda(), _weight(2048, BF, 12).cuda()
    whole, _ = dflash2.sublayer_norm(x, w)
    for i in (0, 150, 300):
        one, _ = dflash2.sublayer_norm(x[i:i + 1], w)
        assert torch.equal(one[0], whole[i])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,cols", [(1, 1), (1, 16), (3, 128), (5, 129), (2, 1000), (17, 1024), (300, 4096)])
def test_quantise(cuda, dtype, n, cols):
    x = ref.rows(n, cols, dtype, 13)
    if cols > 100:
        x[0, :128] = 0
        x[-1, 3] = math.inf
        x[-1, 9] = math.nan
        x[n // 2, 50] = 1e30
    codes, scale = dflash2.quantize_blocks_e4m3(x.cuda())
    want, want_s = ref.quantise_blocks(x.float())
    assert torch.equal(scale.cpu(), want_s) and ref.same_codes(codes, want)


def test_quantise_ties_tiny_blocks_and_strides(cuda):
    vals = ref.e4m3_values()[:127]
    mids = ((vals[:-1] + vals[1:]) / 2).float()
    x = torch.zeros((4, 256))
    x[0, 0], x[0, 1:127] = 448.0, mids                      # every tie at scale 1
    x[1, 128], x[1, 129:255] = -448.0, -mids
    x[2] = torch.linspace(-1, 1, 256) * 2.0 ** -120          # below the floor: codes near zero
    x[3] = torch.linspace(-1, 1, 256) * 2.0 ** -99
    codes, scale = dflash2.quantize_blocks_e4m3(x.cuda())
    want, want_s = ref.quantise_blocks(x)
    assert torch.equal(scale.cpu(), want_s) and ref.same_codes(codes, want)
    wide = torch.zeros((4, 400))
    wide[:, 3:259] = x
    codes2, scale2 = dflash2.quantize_blocks_e4m3(wide.cuda()[:, 3:259])
    assert torch.equal(codes2, codes) and torch.equal(scale2, scale)


def test_no_rows(cuda):
    w = _weight(64, BF, 1).cuda()
    x = torch.empty((0, 64), dtype=BF, device=cuda)
    assert dflash2.sublayer_norm(x, w)[0].shape == (0, 64)
    assert dflash2.sublayer_join(x, x, next_weight=w, e4m3=True)[2].shape == (0, 1)
    assert dflash2.quantize_blocks_e4m3(x)[0].shape == (0, 64)
