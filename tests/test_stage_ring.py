"""The stages of the product kernels, played through on the host: nothing is loaded over a block in use,
and no commit is still to arrive in the shared memory of a CTA that leaves."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("ring") / "stage_ring_check")
    cmd = ["g++", "-std=c++17", "-O2", "-Wall", os.path.join(HERE, "stage_ring_check.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


def _play(program, *args):
    r = subprocess.run([program, *map(str, args)], capture_output=True, text=True, timeout=60)
    return r.returncode, r.stdout


# few rows: one producer in one CTA; many: two, for the even and the odd blocks, in each of two
@pytest.mark.parametrize("producers,ctas", [(1, 1), (2, 2)])
@pytest.mark.parametrize("stages", range(2, 9))
def test_nothing_arrives_after_a_cta_left(program, producers, ctas, stages):
    for blocks in (1, 2, stages - 1, stages, stages + 1, 2 * stages + 1, 37):
        for seed in range(6):
            code, said = _play(program, stages, blocks, producers, ctas, seed, "empty")
            assert code == 0, (stages, blocks, seed, said)


@pytest.mark.parametrize("producers,ctas", [(1, 1), (2, 2)])
def test_waiting_for_the_copies_alone_is_seen(program, producers, ctas):
    """The same with a wait that ends when the last copies have landed."""
    said = [_play(program, 5, 12, producers, ctas, seed, "full") for seed in range(60)]
    assert any(code == 1 and "left" in text for code, text in said), said
