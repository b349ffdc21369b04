"""Norms, block products and rotary positions where offsets pass 32 bits, on two streams at once, and
captured before their first call."""
import os
import subprocess
import sys

import pytest
import torch

import layer_ref as ref
from block_draft_proposal_gb300 import dflash2

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _ends(n):
    return torch.tensor([0, 1, n // 2, n - 2, n - 1])


def test_norm_and_quantise_beyond_32_bits(cuda):
    n, hidden = 270_001, 8000                                  # 2.16e9 values
    x = torch.empty((n, hidden), dtype=BF, device=cuda)
    rows = ref.rows(5, hidden, BF, 1).cuda()
    at = _ends(n).cuda()
    x[at] = rows
    w = torch.ones(hidden, dtype=BF, device=cuda)
    out, _ = dflash2.sublayer_norm(x, w)
    want, _ = dflash2.sublayer_norm(rows, w)
    assert torch.equal(out[at], want)
    r, nxt, _ = dflash2.sublayer_join(x, x, post_weight=w, next_weight=w, residual_out=out)
    want_r, want, _ = dflash2.sublayer_join(rows, rows, post_weight=w, next_weight=w)
    assert torch.equal(r[at], want_r) and torch.equal(nxt[at], want)
    del out, r, nxt
    codes, scale = dflash2.quantize_blocks_e4m3(x)
    want_c, want_s = dflash2.quantize_blocks_e4m3(rows)
    assert torch.equal(codes[at], want_c) and torch.equal(scale[at], want_s)
    codes, scale = dflash2.sublayer_norm(x, w, e4m3=True)
    want_c, want_s = dflash2.sublayer_norm(rows, w, e4m3=True)
    assert torch.equal(codes[at], want_c) and torch.equal(scale[at], want_s)


def test_product_beyond_32_bits(cuda):
    n, n_in, n_out = 950_000, 48, 2304                         # 2.19e9 results
    w_q, w_s = (t.cuda() for t in ref.weights(n_out, n_in, 2))
    x = torch.zeros((n, n_in), dtype=BF, device=cuda)
    at = _ends(n).cuda()
    x[at] = ref.rows(5, n_in, BF, 3).cuda()
    y, err = dflash2.linear_fp8_blocks(x, w_q, w_s)
    x_q, x_s = ref.quantise_blocks(x[at].cpu().float())
    want, bound = ref.product(x_q, x_s, w_q.cpu(), w_s.cpu())
    got = y[at].cpu().double()
    assert int(err) == 0 and bool(((got - want).abs() <= bound + ref.U_BF16 * want.abs()).all())
    assert not y[2:1000].any() and not y[-1000:-2].any()
    # many weights: the few rows' kernel over as many CTAs, its weights' offsets beyond 32 bits
    n_in, n_out = 4096, 540_000                                # 2.2e9 codes
    w_q = torch.zeros((n_out, n_in), dtype=torch.uint8, device=cuda)
    w_s = torch.ones(((n_out + 127) // 128, n_in // 128), device=cuda)
    some, _ = ref.weights(5, n_in, 4)
    at = _ends(n_out)
    w_q[at.cuda()] = some.cuda()
    x = ref.rows(3, n_in, BF, 5)
    y, err = dflash2.linear_fp8_blocks(x.cuda(), w_q, w_s)
    x_q, x_s = ref.quantise_blocks(x.float())
    want, bound = ref.product(x_q, x_s, some, torch.ones((1, n_in // 128)))
    got = y[:, at.cuda()].cpu().double()
    assert int(err) == 0 and bool(((got - want).abs() <= bound + ref.U_BF16 * want.abs()).all())
    assert not y[:, 2:1000].any()


def test_rotary_beyond_32_bits(cuda):
    n, heads, d = 270_001, 64, 128                             # 2.2e9 values
    q = torch.empty((n, heads, d), dtype=BF, device=cuda)
    at = _ends(n).cuda()
    g = torch.Generator().manual_seed(6)
    q[at] = torch.randn((5, heads, d), generator=g).to(BF).cuda()
    pos = torch.arange(n, device=cuda)
    table = dflash2.rotary_table(d)
    out, _, err = dflash2.rotary(q, None, pos, table)
    want, _, _ = dflash2.rotary(q[at].contiguous(), None, pos[at].contiguous(), table)
    assert int(err) == 0 and torch.equal(out[at], want)
    dflash2.rotary(q, None, pos, table, q_out=q)
    assert torch.equal(q[at], want)


def test_two_streams_at_once(cuda):
    """Calls that overlap on the GPU, each with its own buffers, give what they give alone."""
    w_q, w_s = (t.cuda() for t in ref.weights(1500, 2048, 7))
    norm_w = torch.ones(2048, dtype=BF, device=cuda)
    streams = [torch.cuda.Stream() for _ in range(3)]
    xs = [ref.rows(n, 2048, BF, n).cuda() for n in (3, 50, 700)]

    def chain(x, stream):
        r, n, s = dflash2.sublayer_join(x, x, post_weight=norm_w, next_weight=norm_w, e4m3=True, stream=stream)
        y, _ = dflash2.linear_fp8_blocks(n, w_q, w_s, x_scale=s, stream=stream)
        z, err = dflash2.linear_fp8_blocks(x, w_q, w_s, stream=stream)
        return r, y, z, err

    want = [chain(x, None) for x in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        got.append([chain(x, s) for x, s in zip(xs, streams)])
    for s in streams:
        s.synchronize()
    for round_ in got:
        for have, alone in zip(round_, want):
            assert all(torch.equal(a, b) for a, b in zip(have, alone))


SCRIPT = """
import sys, torch
sys.path[:0] = [%r, %r]
import layer_ref as ref
from block_draft_proposal_gb300 import dflash2
torch.cuda.init()
x = [ref.rows(n, 512, torch.bfloat16, n).cuda() for n in (3, 50, 300)]
w_q, w_s = (t.cuda() for t in ref.weights(700, 512, 1))
w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
table = dflash2.rotary_table(64)
pos = torch.arange(300, device="cuda")
slots = torch.arange(300, device="cuda")
cache = dflash2.new_kv_cache(20, 16, 2, 64, e4m3=True)
graph = torch.cuda.CUDAGraph()
def run():
    ys = [dflash2.linear_fp8_blocks(t, w_q, w_s)[0] for t in x]
    r, n, s = dflash2.sublayer_join(x[2], x[2], next_weight=w, e4m3=True)
    z, _ = dflash2.linear_fp8_blocks(n, w_q, w_s, x_scale=s)
    h = x[2].view(300, 8, 64)
    q, k, _ = dflash2.rotary_kv_write(cache, h[:, :4], h[:, 4:6], h[:, 6:], pos, table, slots, with_k=True)
    return ys + [r, n, s, z, q, k]
with torch.cuda.graph(graph):
    captured = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, run()))
print("the same")
"""


def test_captured_before_the_first_call(cuda):
    r = subprocess.run([sys.executable, "-c", SCRIPT % (ROOT, os.path.join(ROOT, "tests"))], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "the same" in r.stdout, r.stderr[-2000:]
