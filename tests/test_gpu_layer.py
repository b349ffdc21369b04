"""One layer's attention as a user runs it: norm, FP8 projection, rotary positions into the cache,
attention of drafted trees, FP8 output projection, and the join with the next norm.  Each stage is
held to its 64-bit form on the stage before's own results; a captured pass replays it."""
import pytest
import torch

import layer_ref as ref
from attention_ref import U_BF16, U_F16, attend, cached_rows, chain_or_tree, check
from block_draft_proposal_gb300 import dflash2

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Layer:
    def __init__(self, hidden, hq, hk, d, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.hidden, self.hq, self.hk, self.d = hidden, hq, hk, d
        self.pre, self.post, self.nxt = ((1 + 0.2 * torch.randn(hidden, generator=g)).to(BF) for _ in range(3))
        self.qkv = ref.weights((hq + 2 * hk) * d, hidden, seed + 1)
        self.out = ref.weights(hidden, hq * d, seed + 2)
        scale = (0.3 / (hidden ** 0.5) for _ in range(2))
        self.qkv, self.out = ((q, s / s.mean() * c / 100) for (q, s), c in zip((self.qkv, self.out), scale))
        self.gate = torch.randn(hidden, generator=g).to(BF)
        self.table = dflash2.rotary_table(d, 1e6, [d // 2 - 2 * (d // 8), d // 8, d // 8], interleaved=False)
        self.dev = {n: getattr(self, n).cuda() for n in ("pre", "post", "nxt", "gate")}
        self.qkv_dev, self.out_dev = ([t.cuda() for t in w] for w in (self.qkv, self.out))

    def run(self, x, cache, positions, slots, table, cu, lens, mask, err, out=None):
        n, hq, hk, d = len(x), self.hq, self.hk, self.d
        s = {}
        s["codes"], s["scale"] = dflash2.sublayer_norm(x, self.dev["pre"], e4m3=True)
        s["qkv"], _ = dflash2.linear_fp8_blocks(s["codes"], *self.qkv_dev, x_scale=s["scale"], err=err)
        q, k, v = s["qkv"].view(n, hq + 2 * hk, d).split([hq, hk, hk], 1)
        s["q"], _, _ = dflash2.rotary_kv_write(cache, q, k, v, positions, self.table, slots, err=err)
        s["attn"], _, _ = dflash2.tree_attention(s["q"], cache, table, cu, lens, d ** -0.5, tree_mask=mask, err=err)
        s["y"], _ = dflash2.linear_fp8_blocks(s["attn"].view(n, hq * d), *self.out_dev, err=err)
        s["r"], s["next"], s["next_scale"] = dflash2.sublayer_join(
            x, s["y"], post_weight=self.dev["post"], gate=self.dev["gate"], gate_act="tanh", branch_scale=0.5,
            next_weight=self.dev["nxt"], e4m3=True, residual_out=out)
        return s


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hidden,hq,hk,d,drafts", [(512, 8, 2, 64, [1, 5, 3]), (1024, 8, 4, 128, [16, 7, 1, 12])])
def test_layer(cuda, hidden, hq, hk, d, drafts, e4m3):
    layer = Layer(hidden, hq, hk, d)
    g = torch.Generator().manual_seed(5)
    ctx, ps = [40, 3, 129, 17][:len(drafts)], 16
    lens = [c + t for c, t in zip(ctx, drafts)]
    per = -(-max(lens) // ps)
    pages = len(drafts) * per
    table = torch.randperm(pages, generator=g).int().view(len(drafts), per)
    cache = dflash2.new_kv_cache(pages, ps, hk, d, e4m3=e4m3)
    err = torch.zeros(1, dtype=torch.int32, device=cuda)

    def slots_of(b, at):
        return [int(table[b, i // ps]) * ps + i % ps for i in at]

    # the contexts first, as one pass whose attention is the prompts' own
    total = sum(ctx)
    x = ref.rows(total, hidden, F32, 6).cuda()
    where = torch.tensor([[i for c in ctx for i in range(c)], [i % 7 for c in ctx for i in range(c)],
                          [i % 5 for c in ctx for i in range(c)]])
    slots = torch.tensor([s for b, c in enumerate(ctx) for s in slots_of(b, range(c))])
    cu = torch.tensor([0, *torch.tensor(ctx).cumsum(0).tolist()], dtype=torch.int32)
    codes, scale = dflash2.sublayer_norm(x, layer.dev["pre"], e4m3=True)
    qkv, _ = dflash2.linear_fp8_blocks(codes, *layer.qkv_dev, x_scale=scale, err=err)
    q, k, v = qkv.view(total, hq + 2 * hk, d).split([hq, hk, hk], 1)
    q, k, _ = dflash2.rotary_kv_write(cache, q, k, v, where.cuda(), layer.table, slots.cuda(), with_k=True, err=err)
    mine, _, _ = dflash2.prompt_attention(q, k, v, cu.cuda(), d ** -0.5, err=err)
    # the same rows as drafted chains over the cache just written
    over, _, _ = dflash2.tree_attention(q, cache, table.cuda(), cu.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(),
                                        d ** -0.5, err=err)
    assert int(err) == 0
    if not e4m3:
        at = 0
        for c in ctx:
            rows = slice(at, at + c)
            want, _, bound, _ = attend(q[rows].cpu().double(), k[rows].cpu().double(), v[rows].cpu().double(),
                                       chain_or_tree(c, 0, None), d ** -0.5, U_BF16, U_BF16)
            check("prompt", mine[rows], want, bound)
            check("over the cache", over[rows], want, bound)
            at += c

    # the drafted trees
    n = sum(drafts)
    x = ref.rows(n, hidden, F32, 7)
    mask = []
    for t in drafts:
        seen = []
        for j in range(t):
            seen.append((1 << j) | (seen[max(0, j - 2)] if j else 0))
        mask += [[s] for s in seen]
    mask = torch.tensor(mask)
    place = torch.tensor([[c + j for c, t in zip(ctx, drafts) for j in range(t)]] * 3)
    slots = torch.tensor([s for b, (c, t) in enumerate(zip(ctx, drafts)) for s in slots_of(b, range(c, c + t))])
    cu = torch.tensor([0, *torch.tensor(drafts).cumsum(0).tolist()], dtype=torch.int32)
    args = [t.cuda() for t in (x, place, slots, table, cu, torch.tensor(lens, dtype=torch.int32), mask)]
    s = layer.run(args[0], cache, *args[1:6], args[6], err)
    assert int(err) == 0

    wide = x.double()
    want, _ = ref.norm(wide, layer.pre.double(), 0.0, 1e-6)
    ref.held_as_blocks(s["codes"], s["scale"], want, ref.NORM * want.abs(), "norm")
    want, bound = ref.product(s["codes"].cpu(), s["scale"].cpu(), *layer.qkv)
    check("projection", s["qkv"], want, bound + U_BF16 * want.abs())
    q, k, v = s["qkv"].cpu().double().view(n, hq + 2 * hk, d).split([hq, hk, hk], 1)
    angle = ref.angles(place, layer.table.freq.cpu(), layer.table.axis.cpu())
    want, bound = ref.turn(q, angle, False)
    check("queries", s["q"], want, bound + U_BF16 * want.abs())
    held = [None if t is None else t.cpu() for t in cache]
    if not e4m3:
        want, bound = ref.turn(k, angle, False)
        got = held[0][slots // ps, :, slots % ps]
        check("keys", got, want, bound + U_BF16 * want.abs())
    at = 0
    for b, (c, t) in enumerate(zip(ctx, drafts)):
        rows = slice(at, at + t)
        keys, vals = cached_rows(held, b, c + t, table)
        want, _, bound, _ = attend(s["q"][rows].cpu().double(), keys, vals, chain_or_tree(t, c, mask[rows]),
                                   d ** -0.5, U_F16 if e4m3 else U_BF16, U_BF16)
        if e4m3:                                           # the queries as two E4M3 parts: eight bits
            size = torch.einsum("thd,nhd->thn", s["q"][rows].cpu().double().abs(),
                                keys.repeat_interleave(hq // hk, 1).abs()).amax(-1) * d ** -0.5
            top = vals.abs().amax()
            bound = bound + (2 * 2.0 ** -8 * size * top)[..., None]
        check(f"attention {b}", s["attn"][rows], want, bound)
        at += t
    a_q, a_s = ref.quantise_blocks(s["attn"].cpu().view(n, hq * d).float())
    want, bound = ref.product(a_q, a_s, *layer.out)
    check("output projection", s["y"], want, bound + U_BF16 * want.abs())
    want_r, dr, want, dout = ref.join(wide, s["y"].cpu().double(), layer.post.double(), layer.gate.double(), "tanh",
                                      0.5, layer.nxt.double(), 0.0, 1e-6)
    check("residual", s["r"], want_r, dr + ref.U_F32 * want_r.abs())
    ref.held_as_blocks(s["next"], s["next_scale"], want, dout, "next norm")

    # captured, and replayed on other hidden states, in place in the residual stream
    stream, where_to = torch.cuda.Stream(), args[0].clone()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.run(where_to, cache, *args[1:6], args[6], err, out=where_to)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = layer.run(where_to, cache, *args[1:6], args[6], err, out=where_to)
    where_to.copy_(args[0])
    graph.replay()
    assert torch.equal(where_to, s["r"]) and torch.equal(again["next"], s["next"]) and int(err) == 0
