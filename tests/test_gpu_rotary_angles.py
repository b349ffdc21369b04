"""Sines and cosines of the rotary positions next to a quarter turn, where one of them is small: held to
0.8 of its own last place, as the slow pairs' at the first positions are."""
import math

import pytest
import torch

from block_draft_proposal_gb300 import dflash2

pytestmark = pytest.mark.gpu


def _exact(phase):
    """(cos, sin) of phase / 2^64 turns in 64 bits: the nearest quarter turn leaves in whole numbers, so that
    what is left is right to 2^-51 of itself."""
    quarter = ((phase >> 61) + 1) >> 1
    rest = (phase - (quarter << 62)) * 2.0 ** -64 * math.tau
    c, s = math.cos(rest), math.sin(rest)
    return ((c, s), (-s, c), (-c, -s), (s, -c))[quarter % 4]


@pytest.mark.parametrize("quarter", [0, 1, 2, 3])
def test_small_sines_and_cosines(cuda, quarter):
    """Frequencies of 2^j and of j random bits beside each quarter turn, and what base 1e7 has in its slowest
    pairs; pairs (1, 0) become (cos, sin)."""
    g = torch.Generator().manual_seed(quarter)
    odd = torch.randint(0, 2 ** 62, (55,), generator=g) >> torch.arange(1, 56)
    slow = dflash2.rotary_table(128, 1e7, device="cpu").freq[-12:]
    freq = torch.cat([torch.ones(61, dtype=torch.int64) << torch.arange(61), odd, slow])
    half = len(freq)
    positions = torch.tensor([-1001, -7, -3, -1, 0, 1, 2, 3, 5, 17, 1000])
    turned = freq + ((quarter if quarter < 2 else quarter - 4) << 62)
    table = dflash2.RotaryTable(turned.to(cuda), torch.zeros(half, dtype=torch.uint8, device=cuda))
    x = torch.zeros((len(positions), 1, 2 * half), device=cuda)
    x[..., :half] = 1
    got, _, err = dflash2.rotary(x, None, positions.to(cuda), table)
    assert int(err) == 0
    got = got[:, 0].cpu().double()
    for i, p in enumerate(positions.tolist()):
        for j, f in enumerate(turned.tolist()):
            phase = (p * f) % 2 ** 64
            for have, want in zip((float(got[i, j]), float(got[i, half + j])), _exact(phase)):
                place = math.ldexp(1.0, math.frexp(want)[1] - 24) if want else 0.0
                assert abs(have - want) <= 0.8 * place + 2.0 ** -50 * abs(want), (p, f, have, want)
