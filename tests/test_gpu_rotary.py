"""Rotary positions on the GPU against 64 bits, and what they write into the cache."""
import math

import pytest
import torch

import layer_ref as ref
from attention_ref import check, e4m3_values
from block_draft_proposal_gb300 import dflash2

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Case:
    def __init__(self, n, hq, hk, d, rot, axes=1, adjacent=False, dtype=BF, seed=0, far=100000, magnitude=1.0):
        g = torch.Generator().manual_seed(seed + n + d)
        self.n, self.hq, self.hk, self.d, self.dtype = n, hq, hk, d, dtype
        qkv = torch.randn((n, hq + 2 * hk, d), generator=g).to(dtype)
        self.packed = qkv.cuda()
        self.q, self.k, self.v = self.packed.split([hq, hk, hk], 1)
        half = rot // 2
        sections = [half - (axes - 1) * (half // (axes + 1))] + [half // (axes + 1)] * (axes - 1)
        self.table = dflash2.rotary_table(rot, 1e4, sections, adjacent=adjacent, magnitude=magnitude)
        self.positions = torch.randint(-far, far, (axes, n), generator=g)
        self.adjacent, self.magnitude = adjacent, magnitude

    def turned(self, x):
        angle = ref.angles(self.positions, self.table.freq.cpu(), self.table.axis.cpu())
        return ref.turn(x.cpu().double(), angle, self.adjacent, self.magnitude)

    def check(self, name, got, x):
        want, bound = self.turned(x)
        check(name, got, want, bound + ref.HALF_STEP[self.dtype] * want.abs() + ref.TINY)


SHAPES = [  # n, q heads, kv heads, head_dim, rotary_dim, axes, adjacent
    (1, 32, 8, 128, 128, 1, False), (5, 4, 1, 64, 64, 3, False), (19, 10, 2, 128, 64, 2, False),
    (3, 8, 8, 256, 256, 1, True), (7, 3, 1, 80, 40, 2, True), (7, 3, 1, 80, 80, 2, False),
    (4, 5, 5, 96, 96, 3, False), (6, 2, 1, 72, 24, 1, True), (2, 1, 1, 2, 2, 1, False),
    (9, 3, 3, 33, 10, 2, False), (9, 3, 3, 33, 10, 2, True), (2, 70, 1, 128, 128, 1, False),
    (300, 4, 2, 16, 16, 1, False),
    # halves that begin at a step of 4, not of 8, and rows of such steps
    (19, 10, 2, 80, 40, 2, False), (7, 3, 1, 72, 72, 3, False), (33, 5, 1, 36, 24, 1, False),
    (3, 4, 4, 252, 248, 1, False), (5, 2, 1, 20, 12, 1, True), (300, 2, 2, 256, 120, 3, False),
    (1, 1, 1, 4, 4, 1, True), (65, 3, 3, 132, 8, 1, False), (2, 70, 1, 100, 72, 1, False)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_turns(cuda, shape, dtype):
    n, hq, hk, d, rot, axes, adjacent = shape
    c = Case(n, hq, hk, d, rot, axes, adjacent, dtype, magnitude=1.25)
    before = c.packed.clone()
    q, k, err = dflash2.rotary(c.q, c.k, c.positions.cuda(), c.table)
    assert int(err) == 0 and torch.equal(c.packed, before)
    c.check("q", q, c.q)
    c.check("k", k, c.k)
    # in place in the packed projection, the values and what is not turned untouched
    q2, k2, _ = dflash2.rotary(c.q, c.k, c.positions.cuda(), c.table, q_out=c.q, k_out=c.k)
    assert torch.equal(c.q, q) and torch.equal(c.k, k) and torch.equal(c.packed[:, hq + hk:], before[:, hq + hk:])
    assert torch.equal(q[..., rot:], before[:, :hq, rot:])
    q3, none, _ = dflash2.rotary(before[:, :hq], None, c.positions.cuda(), c.table)
    assert none is None and torch.equal(q3, q)


def test_turned_back(cuda):
    c = Case(40, 4, 2, 128, 128, 3, dtype=F32)
    q, k, _ = dflash2.rotary(c.q, c.k, c.positions.cuda(), c.table)
    back, _, _ = dflash2.rotary(q, k, -c.positions.cuda(), c.table)
    x = c.q.cpu().double()
    size = torch.hypot(x[..., :64], x[..., 64:]).repeat(1, 1, 2)
    # two turns of vectors of this length, |a| + |b| at most root two of it
    check("back", back, x, 2 * math.sqrt(2) * ref.TURN * 1.01 * size + 2 * ref.U_F32 * size)


@pytest.mark.parametrize("eighths", [False, True])
def test_sines_and_cosines(cuda, eighths):
    """Pairs (1, 0) become (cos, sin): the last rounding's half place, and 0.3 of one for the terms that
    are added to the angle (a ninth of the sine, three roundings in it) and the series' end."""
    c = Case(1000, 1, 1, 256, 256, dtype=F32, far=2 ** 62)
    if eighths:                                                # of a turn, and steps of 2^-8 from there
        c.table = c.table._replace(freq=torch.arange(128, device=cuda) << 56)
        c.positions = torch.arange(-500, 500)[None]
    x = torch.zeros((1000, 1, 256), device=cuda)
    x[..., :128] = 1
    q, _, _ = dflash2.rotary(x, None, c.positions.cuda(), c.table)
    angle = ref.angles(c.positions, c.table.freq.cpu(), c.table.axis.cpu())
    for got, want in ((q[:, 0, :128], torch.cos(angle)), (q[:, 0, 128:], torch.sin(angle))):
        place = torch.ldexp(torch.ones_like(want), torch.frexp(want)[1] - 24)
        # the reference's own angle is rounded: up to pi, to 2^-52
        assert bool(((got.cpu().double() - want).abs() <= 0.8 * place + 2.0 ** -51).all())


def test_far_positions(cuda):
    c = Case(8, 2, 1, 64, 64)
    c.positions = torch.tensor([[0, 1, -1, 2 ** 31, 2 ** 40 + 1, -2 ** 50 + 3, 2 ** 62, -2 ** 63]])
    q, _, _ = dflash2.rotary(c.q, c.k, c.positions.cuda(), c.table)
    c.check("q", q, c.q)


def test_tables(cuda):
    t = dflash2.rotary_table(16, 100.0, [4, 2, 2], interleaved=True, device="cpu")
    assert t.axis.tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    for j, f in enumerate(t.freq.tolist()):
        assert abs(f * 2.0 ** -64 * math.tau - 100.0 ** (-j / 8)) < 1e-15
    t = dflash2.rotary_table(8, inv_freq=[1.0, 7.0, 0.5, -0.25], device="cpu")   # past half a turn; backwards
    for f, want in zip(t.freq.tolist(), [1.0, 7.0, 0.5, -0.25]):
        assert abs(math.remainder(f * 2.0 ** -64 * math.tau - want, math.tau)) < 1e-14


def test_an_axis_that_is_not_there(cuda):
    c = Case(5, 2, 1, 64, 64, axes=2)
    axis = c.table.axis.clone()
    axis[3] = 2
    table = c.table._replace(axis=axis)
    q, _, err = dflash2.rotary(c.q, c.k, c.positions.cuda(), table)
    assert int(err) == dflash2.DEVERR_ID_RANGE
    c.table = table
    c.check("q", q, c.q)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("e4m3", [False, True])
def test_into_the_cache(cuda, shape, dtype, e4m3):
    n, hq, hk, d, rot, axes, adjacent = shape
    c = Case(n, hq, hk, d, rot, axes, adjacent, dtype, seed=3)
    ps = 7
    pages = n // ps + 3
    slots = torch.randperm(pages * ps, generator=torch.Generator().manual_seed(1))[:n]
    if n > 4:
        slots[2], slots[3] = -1, pages * ps                    # skipped; out of range
    cache = dflash2.new_kv_cache(pages, ps, hk, d, dtype=dtype, e4m3=e4m3)
    plain = dflash2.new_kv_cache(pages, ps, hk, d, dtype=dtype, e4m3=e4m3)
    where = (c.positions.cuda(), c.table, slots.cuda())
    q, k, err = dflash2.rotary_kv_write(cache, c.q, c.k, c.v, *where, with_k=True)
    assert int(err) == (dflash2.DEVERR_ID_RANGE if n > 4 else 0)
    q0, k0, _ = dflash2.rotary(c.q, c.k, c.positions.cuda(), c.table)
    assert torch.equal(q, q0) and torch.equal(k, k0)
    dflash2.kv_cache_write(plain, k0, c.v, slots.cuda())
    assert torch.equal(cache.v, plain.v)                       # values: as the write has them
    if e4m3:
        assert torch.equal(cache.v_exp, plain.v_exp)
        want, bound = c.turned(c.k)
        live = (slots >= 0) & (slots < pages * ps)
        at, off = slots[live] // ps, slots[live] % ps
        scale = 2.0 ** (cache.k_exp.cpu()[at, :, off].double() - 127)
        amax = want[live].abs().amax(-1)
        assert bool((amax <= 448 * scale * (1 + 2.0 ** -20)).all())
        assert bool((amax > 224 * scale * (1 - 2.0 ** -20)).all() or d < 8)
        got = e4m3_values()[cache.k.cpu()[at, :, off].long()] * scale[..., None]
        allowed = want[live].abs() * (2.0 ** -4 + 2.0 ** -20) + 2.0 ** -10 * scale[..., None] + 1.1 * bound[live]
        assert bool(((got - want[live]).abs() <= allowed).all())
        untouched = torch.ones((pages, ps), dtype=torch.bool)
        untouched[at, off] = False
        assert not cache.k.cpu().permute(0, 2, 1, 3)[untouched].any()
        if dtype == F32:                                       # nothing is rounded in between
            assert torch.equal(cache.k, plain.k) and torch.equal(cache.k_exp, plain.k_exp)
    else:
        assert torch.equal(cache.k, plain.k)
    again = dflash2.new_kv_cache(pages, ps, hk, d, dtype=dtype, e4m3=e4m3)
    none, none2, _ = dflash2.rotary_kv_write(again, None, c.k, c.v, *where)
    assert none is None and none2 is None and torch.equal(again.k, cache.k) and torch.equal(again.v, cache.v)


@pytest.mark.parametrize("skip", [1, 2, 4, 8])
def test_misaligned_rows_and_one_axis(cuda, skip):
    c = Case(11, 4, 2, 128, 128, dtype=BF)
    flat = torch.zeros(skip + c.q.numel(), dtype=BF, device=cuda)
    odd = flat[skip:].view(11, 4, 128)
    odd.copy_(c.q)
    got, _, _ = dflash2.rotary(odd, None, c.positions[0].contiguous().cuda(), c.table)
    c.check("q", got, c.q)


def test_special_values_stay_in_their_pairs(cuda):
    for adjacent in (False, True):
        c = Case(3, 2, 1, 64, 32, adjacent=adjacent, dtype=F32)
        c.packed[0, 0, 5], c.packed[1, 1, 40] = math.nan, math.inf
        q, _, _ = dflash2.rotary(c.q, c.k, c.positions.cuda(), c.table)
        other = 4 if adjacent else 21
        bad = torch.zeros(q.shape, dtype=torch.bool)
        bad[0, 0, [5, other]] = True
        assert torch.equal(torch.isnan(q).cpu(), bad)
        assert math.isinf(float(q[1, 1, 40])) and int(torch.isinf(q).sum()) == 1


def test_no_tokens_and_graphs(cuda):
    c = Case(0, 4, 2, 64, 64)
    q, k, _ = dflash2.rotary(c.q, c.k, c.positions.cuda(), c.table)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    c = Case(9, 4, 2, 64, 64)
    pos, slots = c.positions.cuda(), torch.arange(9, device=cuda)
    cache = dflash2.new_kv_cache(2, 8, 2, 64)
    err, q = torch.zeros(1, dtype=torch.int32, device=cuda), torch.empty((9, 4, 64), dtype=BF, device=cuda)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dflash2.rotary_kv_write(cache, c.q, c.k, c.v, pos, c.table, slots, q_out=q, err=err)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dflash2.rotary_kv_write(cache, c.q, c.k, c.v, pos, c.table, slots, q_out=q, err=err)
    pos += 77
    slots += 5
    graph.replay()
    want, wk, _ = dflash2.rotary(c.q, c.k, pos, c.table)
    k, v, _ = dflash2.kv_cache_read(cache, slots)
    assert torch.equal(q, want) and torch.equal(k, wk) and torch.equal(v, c.v) and int(err) == 0
