"""Attention over the paged cache and over packed prompts on the GPU against
64-bit definitions, within bounds derived from the arithmetic (attention_ref)."""
import math

import pytest
import torch

import attention_ref as ref
from block_draft_proposal_gb300 import dflash2

pytestmark = pytest.mark.gpu
NAN = float("nan")


def _weights_u(dtype, e4m3):
    return 0.0 if dtype == torch.float32 else ref.U_F16 if e4m3 else ref.U_BF16


def _out_u(dtype):
    return ref.U_F32 if dtype == torch.float32 else ref.U_BF16


def _tree_words(t, words, seed, empty_row=None):
    """Random trees as mask words [t, words]; node `empty_row` sees nothing."""
    g = torch.Generator().manual_seed(seed)
    seen = [0] * t
    for j in range(t):
        parent = int(torch.randint(0, j, (1,), generator=g)) if j else -1
        seen[j] = (seen[parent] if parent >= 0 else 0) | (1 << j)
    if empty_row is not None and empty_row < t:
        seen[empty_row] = 0
    out = torch.zeros((t, words), dtype=torch.int64)
    for j in range(t):
        for w in range(words):
            bits = (seen[j] >> (64 * w)) & (2 ** 64 - 1)
            out[j, w] = bits - 2 ** 64 if bits >= 2 ** 63 else bits
    return out


class Case:
    """A paged problem: inputs on the GPU, copies on the host for the reference."""

    def __init__(self, t, ctx, hq, hk, d, ps, dtype=torch.bfloat16, e4m3=False, words=None,
                 seed=0, garbage=NAN, empty_row=None, q_pad=0, spread=1.0):
        g = torch.Generator().manual_seed(1000 + seed)
        self.t, self.ctx, self.dtype, self.e4m3 = t, ctx, dtype, e4m3
        self.hq, self.hk, self.d, self.ps = hq, hk, d, ps
        self.scale = d ** -0.5
        batch, total = len(t), sum(t)
        lens = [a + b for a, b in zip(t, ctx)]
        per = [-(-n // ps) for n in lens]
        pages = sum(per) + 3
        self.cache = dflash2.new_kv_cache(pages, ps, hk, d, dtype=dtype, e4m3=e4m3)
        # what no request wrote holds garbage
        if e4m3:
            self.cache.k.fill_(0x7F), self.cache.v.fill_(0x7F)
            self.cache.k_exp.fill_(175), self.cache.v_exp.fill_(175)
        else:
            self.cache.k.fill_(garbage), self.cache.v.fill_(garbage)
        order = torch.randperm(pages, generator=g)
        width = max(1, max(per)) + 1
        self.table = torch.full((batch, width), 0, dtype=torch.int32)
        at = 0
        k = torch.randn((sum(lens), hk, d), generator=g) * spread
        v = torch.randn((sum(lens), hk, d), generator=g) * torch.exp(
            torch.randn((sum(lens), 1, 1), generator=g))
        slots = []
        for b, n in enumerate(lens):
            mine = order[at:at + per[b]]
            self.table[b, :per[b]] = mine.int()
            line = torch.arange(n)
            slots.append(mine[line // ps] * ps + line % ps if n else line)
            at += per[b]
        self.slots = torch.cat(slots)
        self.k_rows, self.v_rows = k.to(dtype), v.to(dtype)
        self.write()
        wide = torch.randn((total, hq + q_pad, d), generator=g) * 1.5
        self.q_host = wide[:, :hq].to(dtype)
        self.q = wide.to(dtype).cuda()[:, :hq]
        self.cu = torch.tensor([0] + list(torch.tensor(t).cumsum(0)), dtype=torch.int32)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.mask = None
        if words is not None:
            self.mask = torch.cat([_tree_words(n, words, seed * 77 + i, empty_row)
                                   for i, n in enumerate(t)]) if total else \
                torch.zeros((0, words), dtype=torch.int64)

    def write(self):
        dflash2.kv_cache_write(self.cache, self.k_rows.cuda(), self.v_rows.cuda(), self.slots.cuda())

    def run(self, with_lse=True, **kw):
        kw.setdefault("tree_mask", None if self.mask is None else self.mask.cuda())
        return dflash2.tree_attention(self.q, self.cache, self.table.cuda(), self.cu.cuda(),
                                      self.lens.cuda(), self.scale, with_lse=with_lse, **kw)

    def host_cache(self):
        return [None if x is None else x.cpu() for x in self.cache]

    def check(self, out, lse, only=None):
        host = self.host_cache()
        row = 0
        for b, t in enumerate(self.t):
            rows = slice(row, row + t)
            row += t
            if t == 0 or (only is not None and b not in only):
                continue
            k, v = ref.cached_rows(host, b, t + self.ctx[b], self.table)
            seen = ref.chain_or_tree(t, self.ctx[b], None if self.mask is None else self.mask[rows])
            want, wl, bound, lb = ref.attend(self.q_host[rows].double(), k, v, seen, self.scale,
                                             _weights_u(self.dtype, self.e4m3), _out_u(self.dtype))
            ref.check(f"out of request {b}", out[rows], want, bound)
            if lse is not None:
                ref.check(f"lse of request {b}", lse[rows], wl, lb)


BF, F32 = torch.bfloat16, torch.float32
PAGED = [
    # t, ctx, q heads, kv heads, head_dim, page
    ([1], [0], 1, 1, 128, 16),
    ([1, 1, 1], [0, 1, 300], 8, 2, 128, 16),
    ([1], [1000], 32, 8, 128, 16),
    ([1] * 7, [127, 128, 129, 255, 256, 5, 700], 8, 1, 64, 64),
    ([16, 16], [100, 513], 8, 2, 128, 16),
    ([3, 0, 12, 1], [40, 9, 0, 257], 10, 2, 128, 32),
    ([64, 33], [190, 900], 16, 4, 128, 128),
    ([65, 130], [64, 500], 4, 2, 64, 16),
    ([40], [3000], 24, 2, 128, 256),              # 480 rows: two row blocks
    ([5, 9], [130, 77], 7, 1, 128, 16),
    ([128], [0], 2, 2, 64, 32),
    ([2, 2], [20000, 31], 4, 1, 128, 64),         # one request's keys over all SMs
]
GENERAL = [
    ([3, 1], [50, 200], 4, 2, 80, 16),
    ([2, 5], [33, 129], 3, 1, 256, 5),
    ([7], [70], 2, 2, 33, 1),
    ([9, 1], [64, 64], 6, 3, 128, 24),
    ([4], [300], 4, 4, 96, 64),
    ([1], [5], 1, 1, 1, 2),
]


@pytest.mark.parametrize("e4m3", [False, True], ids=["native", "e4m3"])
@pytest.mark.parametrize("words", [None, 2], ids=["chain", "tree"])
@pytest.mark.parametrize("i", range(len(PAGED)))
def test_paged_bf16(cuda, i, words, e4m3):
    if words and max(PAGED[i][0]) > 128:
        words = 3
    c = Case(*PAGED[i], e4m3=e4m3, words=words, seed=i, q_pad=i % 3,
             empty_row=2 if words else None)
    out, lse, err = c.run()
    assert int(err) == 0
    c.check(out, lse)


@pytest.mark.parametrize("e4m3", [False, True], ids=["native", "e4m3"])
@pytest.mark.parametrize("words", [None, 1], ids=["chain", "tree"])
@pytest.mark.parametrize("i", [0, 1, 4, 5, 9])
def test_paged_f32(cuda, i, words, e4m3):
    c = Case(*PAGED[i], dtype=F32, e4m3=e4m3, words=words, seed=50 + i, empty_row=1 if words else None)
    out, lse, err = c.run()
    assert int(err) == 0
    c.check(out, lse)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("e4m3", [False, True], ids=["native", "e4m3"])
@pytest.mark.parametrize("i", range(len(GENERAL)))
def test_paged_any_shape(cuda, i, dtype, e4m3):
    c = Case(*GENERAL[i], dtype=dtype, e4m3=e4m3, words=1 if i % 2 else None, seed=90 + i)
    out, lse, err = c.run()
    assert int(err) == 0
    c.check(out, lse)


@pytest.mark.parametrize("dtype,e4m3", [(BF, False), (BF, True), (F32, False)])
def test_masked_nodes_may_hold_anything(cuda, dtype, e4m3):
    """A node that some rows do not see holds NaN or infinite keys and values:
    those rows keep their results, the rows that see it get NaN or the
    infinity."""
    for bad in (NAN, math.inf, -math.inf):
        c = Case([12, 12], [140, 3], 8, 2, 128, 16, dtype=dtype, e4m3=e4m3, words=1, seed=7)
        clean, clean_lse, _ = c.run()
        start = 140 + 5                                  # node 5 of request 0
        c.v_rows[start] = bad
        c.write()
        out, lse, err = c.run()
        assert int(err) == 0
        assert torch.equal(lse, clean_lse)               # values do not enter the lse
        c.check(out, lse)
        sees = ((c.mask[:12, 0] >> 5) & 1).bool()
        assert sees.any() and not sees.all()
        assert torch.equal(out[:12][~sees], clean[:12][~sees])
        assert torch.equal(out[12:], clean[12:])
        if not e4m3 or math.isnan(bad):
            assert not torch.isfinite(out[:12][sees]).any()
        c.k_rows[start] = NAN                            # its key too
        c.write()
        out, lse, err = c.run()
        assert torch.equal(out[:12][~sees], clean[:12][~sees])
        assert torch.equal(lse[:12][~sees], clean_lse[:12][~sees])
        assert torch.isnan(out[:12][sees]).all() and torch.isnan(lse[:12][sees]).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_that_see_nothing(cuda, e4m3):
    c = Case([5], [0], 4, 2, 128, 16, e4m3=e4m3, words=1, seed=3)
    c.mask[:] = torch.tensor([[0], [1], [0], [4], [0]])
    out, lse, err = c.run()
    for i in (0, 2, 4):
        assert not out[i].any() and torch.isneginf(lse[i]).all()
    v = ref.cached_rows(c.host_cache(), 0, 5, c.table)[1]
    # node 1 sees node 0 alone, node 3 node 2 alone: their values come back
    for i, j in ((1, 0), (3, 2)):
        want = v[j].repeat_interleave(2, 0)
        assert (out[i].double().cpu() - want).abs().max() <= 2 * ref.U_BF16 * want.abs().max()


@pytest.mark.parametrize("e4m3", [False, True])
def test_large_logits_and_wide_values(cuda, e4m3):
    """Logits of several hundred (one key takes all the weight) and values whose
    magnitudes span 2^40 from key to key."""
    c = Case([16, 3], [333, 700], 8, 2, 128, 16, e4m3=e4m3, seed=21, spread=12.0)
    g = torch.Generator().manual_seed(5)
    c.v_rows = (c.v_rows.float() * torch.exp2(torch.randint(-20, 20, (c.v_rows.shape[0], 1, 1),
                                                           generator=g).float())).bfloat16()
    c.write()
    out, lse, err = c.run()
    assert int(err) == 0
    c.check(out, lse)


def test_zero_scale_and_negative_scale(cuda):
    c = Case([4, 1], [200, 150], 4, 2, 128, 16, seed=31)
    for scale in (0.0, -0.1):
        c.scale = scale
        out, lse, _ = c.run()
        c.check(out, lse)


@pytest.mark.parametrize("e4m3", [False, True])
def test_same_bits_every_time_and_on_another_stream(cuda, e4m3):
    c = Case([16] * 5 + [40], [900, 10, 3000, 129, 64, 5000], 16, 4, 128, 32, e4m3=e4m3, words=1,
             seed=41)
    out, lse, _ = c.run()
    ws = torch.empty(dflash2.tree_attention_workspace_size(sum(c.t), 6, 16, 4, 128),
                     dtype=torch.uint8, device=cuda).fill_(0xFF)      # NaN left in the workspace
    s = torch.cuda.Stream()
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    args = (c.q, c.cache, c.table.cuda(), c.cu.cuda(), c.lens.cuda(), c.scale)
    mask = c.mask.cuda()
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        dflash2.tree_attention(*args, tree_mask=mask, out=o2, lse=l2, workspace=ws, err=err, stream=s)
        s.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2) and int(err) == 0


def test_in_a_captured_graph(cuda):
    c = Case([16, 2], [300, 900], 8, 2, 128, 16, seed=61)
    args = (c.q, c.cache, c.table.cuda(), c.cu.cuda(), c.lens.cuda(), c.scale)
    ws = torch.empty(dflash2.tree_attention_workspace_size(18, 2, 8, 2, 128), dtype=torch.uint8,
                     device=cuda)
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    out = torch.empty((18, 8, 128), dtype=BF, device=cuda)
    want, _, _ = dflash2.tree_attention(*args)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dflash2.tree_attention(*args, out=out, workspace=ws, err=err)
    lens = args[4]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    lens[1] -= 100                      # the graph reads the lengths on the device
    want2, _, _ = dflash2.tree_attention(*args)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2) and not torch.equal(want, want2)


@pytest.mark.parametrize("d,ps", [(128, 16), (80, 16)])
def test_data_that_cannot_be_processed(cuda, d, ps):
    def fresh():
        return Case([3, 2], [40, 60], 4, 2, d, ps, seed=71, garbage=1.0)

    c = fresh()
    good, good_lse, _ = c.run()
    c.lens[0] = 2                                         # fewer keys than tokens
    out, lse, err = c.run()
    assert int(err) == dflash2.DEVERR_ID_RANGE
    assert not out[:3].any() and torch.isneginf(lse[:3]).all() and torch.equal(out[3:], good[3:])
    c = fresh()
    c.lens[1] = 10 ** 6                                   # beyond the page table
    out, lse, err = c.run()
    assert int(err) == dflash2.DEVERR_ID_RANGE
    assert not out[3:].any() and torch.isneginf(lse[3:]).all() and torch.equal(out[:3], good[:3])
    for page in (-1, 10 ** 6):                            # a page that is not there: zero rows
        c = fresh()
        c.table[1, 1] = page
        out, lse, err = c.run()
        assert int(err) == dflash2.DEVERR_ID_RANGE
        c2 = fresh()
        slots = c2.slots[43:].clone()                     # request 1's rows, its second page zeroed
        k, v = c2.k_rows.clone(), c2.v_rows.clone()
        k[43 + ps:43 + 2 * ps] = 0
        v[43 + ps:43 + 2 * ps] = 0
        c2.k_rows, c2.v_rows = k, v
        c2.write()
        out2, lse2, _ = c2.run()
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
    c = fresh()
    c.mask = torch.ones((5, 1), dtype=torch.int64)
    out, lse, err = c.run()
    assert int(err) == 0
    c = fresh()
    c.cu[2] = 9                                           # past the packed tokens: clamped
    out, lse, err = c.run()
    assert int(err) == dflash2.DEVERR_ID_RANGE and torch.equal(out, good)


def test_long_context_beyond_32_bit_element_offsets(cuda):
    # pages past element 2^31 of the cache arrays
    hk, d, ps = 16, 128, 64
    pages = 2 ** 31 // (hk * d * ps) + 40
    cache = dflash2.KVCache(*(torch.empty((pages, hk, ps, d), dtype=BF, device=cuda)
                              for _ in range(2)))
    small = dflash2.new_kv_cache(20, ps, hk, d)
    x, y = (torch.randn((1200, hk, d), device=cuda).to(BF) for _ in range(2))
    line = torch.arange(1200, device=cuda)
    dflash2.kv_cache_write(small, x, y, line)
    dflash2.kv_cache_write(cache, x, y, line + (pages - 20) * ps)
    q = torch.randn((4, 32, d), device=cuda).to(BF)
    cu = torch.tensor([0, 4], dtype=torch.int32, device=cuda)
    lens = torch.tensor([1200], dtype=torch.int32, device=cuda)
    table = torch.arange(20, dtype=torch.int32, device=cuda)[None]
    a, _, _ = dflash2.tree_attention(q, small, table, cu, lens, 0.1)
    b, _, _ = dflash2.tree_attention(q, cache, table + (pages - 20), cu, lens, 0.1)
    assert torch.equal(a, b)


def test_many_requests(cuda):
    t = [(i * 7) % 4 for i in range(700)]
    ctx = [(i * 37) % 211 for i in range(700)]
    c = Case(t, ctx, 4, 2, 64, 16, seed=81)
    out, lse, err = c.run()
    assert int(err) == 0
    c.check(out, lse, only=set(range(0, 700, 23)) | {699})


# ---- packed prompts ---------------------------------------------------------------------

def _prompt(lens, hq, hk, d, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    n = sum(lens)
    qkv = torch.randn((n, hq + 2 * hk + pad, d), generator=g)
    qkv[:, :hq] *= 1.5
    qkv = qkv.to(dtype)
    dev = qkv.cuda()
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    return (dev[:, :hq], dev[:, hq:hq + hk], dev[:, hq + hk:hq + 2 * hk]), qkv, cu


def _check_prompt(lens, hq, hk, qkv, out, lse, scale, dtype, only=None):
    at = 0
    for b, n in enumerate(lens):
        rows = slice(at, at + n)
        at += n
        if n == 0 or (only is not None and b not in only):
            continue
        q, k, v = (x.double() for x in (qkv[rows, :hq], qkv[rows, hq:hq + hk],
                                         qkv[rows, hq + hk:hq + 2 * hk]))
        seen = ref.chain_or_tree(n, 0, None)
        want, wl, bound, lb = ref.attend(q, k, v, seen, scale, _weights_u(dtype, False), _out_u(dtype))
        ref.check(f"out of prompt {b}", out[rows], want, bound)
        if lse is not None:
            ref.check(f"lse of prompt {b}", lse[rows], wl, lb)


PROMPTS = [
    ([1], 1, 1, 128), ([1, 1, 2], 8, 2, 128), ([127, 128, 129], 4, 1, 128), ([300], 4, 4, 64),
    ([5, 0, 700, 31], 10, 2, 128), ([64, 65, 63, 1, 17], 8, 8, 64), ([1000], 8, 1, 128),
    ([257, 255], 14, 2, 64), ([33, 90], 6, 3, 96), ([40], 2, 1, 256), ([77], 3, 1, 20),
    ([390], 24, 1, 128),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(PROMPTS)))
def test_prompts(cuda, i, dtype):
    lens, hq, hk, d = PROMPTS[i]
    qkv_dev, qkv, cu = _prompt(lens, hq, hk, d, dtype, 200 + i, pad=i % 2)
    out, lse, err = dflash2.prompt_attention(*qkv_dev, cu.cuda(), d ** -0.5, with_lse=True)
    assert int(err) == 0
    _check_prompt(lens, hq, hk, qkv, out, lse, d ** -0.5, dtype)
    again, _, _ = dflash2.prompt_attention(*qkv_dev, cu.cuda(), d ** -0.5)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_later_tokens_may_hold_anything(cuda, dtype):
    lens, hq, hk, d = [200, 150], 4, 2, 128
    (q, k, v), qkv, cu = _prompt(lens, hq, hk, d, dtype, 300)
    clean, _, _ = dflash2.prompt_attention(q, k, v, cu.cuda(), 0.1)
    for bad in (NAN, math.inf):
        kk, vv = k.clone(), v.clone()
        kk[170], vv[170] = NAN, bad                      # token 170 of prompt 0
        out, _, _ = dflash2.prompt_attention(q, kk, vv, cu.cuda(), 0.1)
        assert torch.equal(out[:170], clean[:170]) and torch.equal(out[200:], clean[200:])
        assert torch.isnan(out[170:200]).all()
        vv2 = v.clone()
        vv2[200, 0, 3] = bad                             # one value, in prompt 1's first token
        out, _, _ = dflash2.prompt_attention(q, k, vv2, cu.cuda(), 0.1)
        assert torch.equal(out[:200], clean[:200])
        assert not torch.isfinite(out[200:, :2, 3]).any()
        keep = torch.ones(d, dtype=torch.bool)
        keep[3] = False
        assert torch.isfinite(out[200:, :2][..., keep]).all() and torch.equal(out[200:, 2:], clean[200:, 2:])


def test_many_prompts_and_misaligned_rows(cuda):
    lens = [(i * 13) % 40 for i in range(600)]
    qkv_dev, qkv, cu = _prompt(lens, 4, 2, 64, BF, 400)
    out, lse, err = dflash2.prompt_attention(*qkv_dev, cu.cuda(), 0.125, with_lse=True)
    assert int(err) == 0
    _check_prompt(lens, 4, 2, qkv, out, lse, 0.125, BF, only=set(range(0, 600, 29)) | {599})
    n, hq, hk, d = 50, 2, 1, 64
    flat = torch.randn(1 + n * (hq + 2 * hk) * d).bfloat16()
    odd = flat.cuda()[1:].view(n, hq + 2 * hk, d)        # rows off 16-byte alignment
    out, _, _ = dflash2.prompt_attention(odd[:, :hq], odd[:, hq:hq + hk], odd[:, hq + hk:],
                                         torch.tensor([0, n], dtype=torch.int32).cuda(), 0.125)
    _check_prompt([n], hq, hk, flat[1:].view(n, hq + 2 * hk, d), out, None, 0.125, BF)


def test_prompt_then_cache_then_next_block(cuda):
    """A prompt's rows equal those of the same tokens taken as one drafted chain
    over the cache they were written to (native cache: the same values)."""
    lens, hq, hk, d, ps = [150], 8, 2, 128, 16
    (q, k, v), qkv, cu = _prompt(lens, hq, hk, d, BF, 500)
    a, la, _ = dflash2.prompt_attention(q, k, v, cu.cuda(), 0.1, with_lse=True)
    cache = dflash2.new_kv_cache(12, ps, hk, d)
    dflash2.kv_cache_write(cache, k, v, torch.arange(150, device=cuda))
    table = torch.arange(12, dtype=torch.int32, device=cuda)[None]
    b, lb, _ = dflash2.tree_attention(q, cache, table, cu.cuda(),
                                      torch.tensor([150], dtype=torch.int32, device=cuda), 0.1,
                                      with_lse=True)
    diff = (a.double() - b.double()).abs()
    assert float((diff - 4 * ref.U_BF16 * 2 * a.double().abs().amax()).max()) <= 0
    assert float((la - lb).abs().max()) <= 1e-4
