"""The paged cache on the GPU: rows land in their slots and nowhere else, E4M3
codes and exponents are the definition's bit for bit, and rows read back are
the values held."""
import math

import pytest
import torch

from attention_ref import e4m3_values, quantise
from block_draft_proposal_gb300 import dflash2

pytestmark = pytest.mark.gpu


def _rows(n, heads, d, dtype, seed, special=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, heads, d), generator=g) * torch.exp2(
        torch.randint(-12, 12, (n, heads, 1), generator=g).float())
    if special and n >= 6:
        x[0] = 0.0
        x[1, 0, 0] = -0.0
        x[2] = 0.0
        x[2, 0, d - 1] = 448.0                   # exactly the largest code at e = 0
        x[3] *= 2.0 ** -70                       # below the exponent range: codes near zero
        x[4] = 2.0 ** 60                         # above it: saturates
        x[5, 0, d // 2] = math.inf
        x[5, heads - 1, 0] = math.nan
    return x.to(dtype)


def _slots(n, pages, ps, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(pages * ps, generator=g)[:n]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,heads,d,ps", [(1, 1, 128, 16), (37, 8, 128, 16), (50, 3, 64, 1),
                                          (41, 2, 256, 64), (33, 5, 80, 7), (9, 1, 1, 3)])
def test_write_then_read(cuda, dtype, e4m3, n, heads, d, ps):
    pages = n // ps + 5
    packed_k, packed_v = _rows(n, heads, d, dtype, 1), _rows(n, heads, d, dtype, 2)
    slots = _slots(n, pages, ps, 3)
    skip = n > 8
    if skip:
        slots[7] = -1
    cache = dflash2.new_kv_cache(pages, ps, heads, d, dtype=dtype, e4m3=e4m3)
    before = [None if t is None else t.clone() for t in cache]
    err = dflash2.kv_cache_write(cache, packed_k.cuda(), packed_v.cuda(), slots.cuda())
    k, v, err2 = dflash2.kv_cache_read(cache, slots.cuda(), dtype=dtype)
    torch.cuda.synchronize()
    assert int(err) == 0 and int(err2) == 0
    live = slots >= 0
    page, off = slots[live] // ps, slots[live] % ps
    for src, held, exps, old, old_e, got in (
            (packed_k, cache.k, cache.k_exp, before[0], before[2], k),
            (packed_v, cache.v, cache.v_exp, before[1], before[3], v)):
        want = old.cpu().clone()
        rows = src[live].double()
        if e4m3:
            codes, e = quantise(rows.reshape(-1, d))
            want[page, :, off] = codes.view(-1, heads, d)
            # a NaN keeps no sign; compare codes with NaN made one code
            nan = (held.cpu() & 127) == 127
            assert torch.equal(nan, (want & 127) == 127)
            assert torch.equal(held.cpu()[~nan], want[~nan])
            want_e = old_e.cpu().clone()
            want_e[page, :, off] = e.view(-1, heads)
            assert torch.equal(exps.cpu(), want_e)
            value = (e4m3_values()[codes.long()] * 2.0 ** (e.double() - 127)[:, None]).view(-1, heads, d)
        else:
            want[page, :, off] = src[live]
            as_bits = {torch.bfloat16: torch.int16, torch.float32: torch.int32}[dtype]
            assert torch.equal(held.cpu().view(as_bits), want.view(as_bits))
            value = rows
        full = torch.zeros((n, heads, d), dtype=torch.float64)
        full[live] = value
        got = got.cpu().double()
        assert torch.equal(torch.isnan(got), torch.isnan(full))
        assert torch.equal(got.nan_to_num(0.0), full.nan_to_num(0.0))


def test_every_code_reads_as_its_value(cuda):
    cache = dflash2.new_kv_cache(3, 16, 1, 64, e4m3=True)
    codes = torch.arange(256, dtype=torch.uint8).view(4, 64)
    cache.k.view(-1, 64)[5:9] = codes.cuda()
    cache.v.view(-1, 64)[5:9] = codes.flip(0).cuda()
    exps = torch.tensor([79, 127, 175, 100], dtype=torch.uint8)
    cache.k_exp.view(-1)[5:9] = exps.cuda()
    cache.v_exp.view(-1)[5:9] = exps.cuda()
    slots = torch.arange(5, 9, device=cuda)
    for dtype in (torch.bfloat16, torch.float32):
        k, v, _ = dflash2.kv_cache_read(cache, slots, dtype=dtype)
        scale = 2.0 ** (exps.double() - 127)[:, None]
        for got, c in ((k, codes), (v, codes.flip(0))):
            want = e4m3_values()[c.long()] * scale
            got = got.cpu().double().view(4, 64)
            assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


def test_rounding_ties_and_boundaries_of_the_exponent(cuda):
    vals = e4m3_values()[:127]
    mids = (vals[:-1] + vals[1:]) / 2                      # every tie at e = 0
    x = torch.cat([mids, vals, torch.tensor([448.0, 449.0, 447.0])]).float()
    rows = torch.zeros((256, 1, 128))
    for i in range(256):
        rows[i, 0, 0] = 448.0
        rows[i, 0, 1] = x[i % x.numel()]
        rows[i, 0, 2] = -x[(7 * i) % x.numel()]
    rows[1, 0, 0] = 448.0 + 2.0 ** -15                     # just above: e = 1
    cache = dflash2.new_kv_cache(16, 16, 1, 128, e4m3=True)
    slots = torch.arange(256, device=cuda)
    dflash2.kv_cache_write(cache, rows.cuda(), rows.cuda(), slots)
    codes, e = quantise(rows.double().view(-1, 128))
    assert torch.equal(cache.k_exp.cpu().view(-1), e)
    assert torch.equal(cache.k.cpu().view(-1, 128), codes)


def test_strided_and_misaligned_inputs(cuda):
    n, heads, d = 19, 2, 128
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn((n, 3 * heads, d), generator=g).bfloat16().cuda()
    flat = torch.randn(1 + n * heads * d, generator=g).bfloat16().cuda()
    odd = flat[1:].view(n, heads, d)                       # rows off 16-byte alignment
    slots = _slots(n, 4, 8, 5).cuda()
    for e4m3 in (False, True):
        cache = dflash2.new_kv_cache(4, 8, heads, d, e4m3=e4m3)
        plain = dflash2.new_kv_cache(4, 8, heads, d, e4m3=e4m3)
        for k, v in ((qkv[:, :heads], qkv[:, heads:2 * heads]), (odd, qkv[:, 2 * heads:])):
            dflash2.kv_cache_write(cache, k, v, slots)
            dflash2.kv_cache_write(plain, k.contiguous(), v.contiguous(), slots)
            for a, b in zip(cache, plain):
                assert a is None or torch.equal(a, b)


def test_read_and_written_again_e4m3_rows_keep_their_values(cuda):
    n, heads, d = 300, 4, 128
    x, y = (_rows(n, heads, d, torch.bfloat16, s, special=False).cuda() for s in (6, 7))
    cache = dflash2.new_kv_cache(40, 16, heads, d, e4m3=True)
    src = _slots(n, 20, 16, 8).cuda()
    dst = (_slots(n, 20, 16, 9) + 320).cuda()
    dflash2.kv_cache_write(cache, x, y, src)
    k, v, _ = dflash2.kv_cache_read(cache, src)
    dflash2.kv_cache_write(cache, k, v, dst)
    k2, v2, _ = dflash2.kv_cache_read(cache, dst)
    assert torch.equal(k, k2) and torch.equal(v, v2)


def test_bad_slots_are_reported_and_touch_nothing(cuda):
    x = torch.randn(4, 2, 64, device=cuda).bfloat16()
    for d_x in (x, x[..., :40].contiguous()):
        cache = dflash2.new_kv_cache(2, 16, 2, d_x.shape[-1])
        slots = torch.tensor([0, 32, 2 ** 40, -5], device=cuda)
        err = dflash2.kv_cache_write(cache, d_x, d_x, slots)
        k, v, err2 = dflash2.kv_cache_read(cache, slots)
        torch.cuda.synchronize()
        assert int(err) == dflash2.DEVERR_ID_RANGE and int(err2) == dflash2.DEVERR_ID_RANGE
        assert torch.equal(k[0], d_x[0]) and not k[1:].any() and not v[1:].any()
        assert torch.equal(cache.k[0, :, 0], d_x[0]) and int((cache.k != 0).sum()) == int((d_x[0] != 0).sum())


def test_many_rows_and_another_stream(cuda):
    n, heads, d, ps = 20000, 8, 128, 32
    g = torch.Generator(device="cuda").manual_seed(10)
    k = torch.randn((n, heads, d), generator=g, device=cuda).bfloat16()
    v = torch.randn((n, heads, d), generator=g, device=cuda).bfloat16()
    pages = n // ps + 1
    slots = torch.randperm(pages * ps, device=cuda)[:n]
    cache = dflash2.new_kv_cache(pages, ps, heads, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        k_out, v_out = torch.empty_like(k), torch.empty_like(v)
        err = torch.zeros(1, dtype=torch.int32, device=cuda)
    dflash2.kv_cache_write(cache, k, v, slots, err=err, stream=s)
    dflash2.kv_cache_read(cache, slots, k_out=k_out, v_out=v_out, err=err, stream=s)
    s.synchronize()
    assert int(err) == 0 and torch.equal(k, k_out) and torch.equal(v, v_out)


def test_slots_beyond_32_bit_element_offsets(cuda):
    # 2^31 elements are passed at page 65536 of 16 x 16 x 128
    heads, d, ps = 16, 128, 16
    pages = 2 ** 31 // (heads * d * ps) + 5
    cache = dflash2.KVCache(*(torch.empty((pages, heads, ps, d), dtype=torch.uint8, device=cuda)
                              for _ in range(2)),
                            *(torch.empty((pages, heads, ps), dtype=torch.uint8, device=cuda)
                              for _ in range(2)))
    x = torch.randn((3, heads, d), device=cuda).bfloat16()
    slots = torch.tensor([pages * ps - 1, 3, (pages - 2) * ps], device=cuda)
    dflash2.kv_cache_write(cache, x, x, slots)
    small = dflash2.new_kv_cache(1, 16, heads, d, e4m3=True)
    dflash2.kv_cache_write(small, x, x, torch.arange(3, device=cuda))
    want, _, _ = dflash2.kv_cache_read(small, torch.arange(3, device=cuda))
    k, v, err = dflash2.kv_cache_read(cache, slots)
    assert int(err) == 0 and torch.equal(k, want) and torch.equal(v, want)
