"""The cache and attention entry points reject bad arguments on the host, before
any CUDA call; workspace sizes are host arithmetic.  No compute call is made."""
import ctypes

import pytest

P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(257)
OK, INVALID, DTYPE, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build_library()
    from block_draft_proposal_gb300 import dflash2
    return dflash2.library()


def _write(lib, **kw):
    a = dict(k=P, v=P, ks=1024, vs=1024, slots=P, n=4, heads=8, d=128, ps=16, pages=10, dtype=1,
             fmt=0, kc=P, vc=P, ke=None, ve=None, err=P)
    a.update(kw)
    return lib.dflash2_kv_cache_write(a["k"], a["v"], a["ks"], a["vs"], a["slots"], a["n"],
                                      a["heads"], a["d"], a["ps"], a["pages"], a["dtype"], a["fmt"],
                                      a["kc"], a["vc"], a["ke"], a["ve"], a["err"], None)


def _read(lib, **kw):
    a = dict(kc=P, vc=P, ke=None, ve=None, slots=P, n=4, heads=8, d=128, ps=16, pages=10, dtype=1,
             fmt=0, k=P, v=P, err=P)
    a.update(kw)
    return lib.dflash2_kv_cache_read(a["kc"], a["vc"], a["ke"], a["ve"], a["slots"], a["n"],
                                     a["heads"], a["d"], a["ps"], a["pages"], a["dtype"], a["fmt"],
                                     a["k"], a["v"], a["err"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), DTYPE), (dict(fmt=2), DTYPE), (dict(d=0), INVALID), (dict(d=257), INVALID),
    (dict(heads=0), INVALID), (dict(ps=0), INVALID), (dict(pages=-1), INVALID), (dict(n=-1), INVALID),
    (dict(n=2 ** 27), INVALID), (dict(pages=2 ** 60), INVALID), (dict(slots=None), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(fmt=1), INVALID),
    (dict(fmt=1, ke=P), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(k=ODD), MISALIGNED), (dict(kc=ODD), MISALIGNED), (dict(slots=ctypes.c_void_p(260)), MISALIGNED),
    (dict(err=ODD), MISALIGNED), (dict(n=0, slots=None, k=None, v=None), OK),
])
def test_cache_refusals(lib, kw, status):
    assert _write(lib, **kw) == status
    assert _read(lib, **kw) == status


def test_write_refuses_overlapping_rows(lib):
    assert _write(lib, ks=1023) == INVALID
    assert _write(lib, vs=-1024) == INVALID


def _tree(lib, **kw):
    a = dict(q=P, qs=4096, kc=P, vc=P, ke=None, ve=None, table=P, width=8, pages=64, ps=16, cu=P,
             lens=P, mask=None, words=0, batch=2, total=32, hq=32, hk=8, d=128, scale=0.1, dtype=1,
             fmt=0, out=P, lse=None, ws=P, bytes=1 << 40, err=P)
    a.update(kw)
    return lib.dflash2_tree_attention(a["q"], a["qs"], a["kc"], a["vc"], a["ke"], a["ve"], a["table"],
                                      a["width"], a["pages"], a["ps"], a["cu"], a["lens"], a["mask"],
                                      a["words"], a["batch"], a["total"], a["hq"], a["hk"], a["d"],
                                      ctypes.c_float(a["scale"]), a["dtype"], a["fmt"], a["out"],
                                      a["lse"], a["ws"], a["bytes"], a["err"], None)


def _prompt(lib, **kw):
    a = dict(q=P, k=P, v=P, qs=4096, ks=1024, vs=1024, cu=P, batch=2, total=32, hq=32, hk=8, d=128,
             scale=0.1, dtype=1, out=P, lse=None, ws=P, bytes=1 << 40, err=P)
    a.update(kw)
    return lib.dflash2_prompt_attention(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["cu"],
                                        a["batch"], a["total"], a["hq"], a["hk"], a["d"],
                                        ctypes.c_float(a["scale"]), a["dtype"], a["out"], a["lse"],
                                        a["ws"], a["bytes"], a["err"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), DTYPE), (dict(hq=30), INVALID), (dict(hk=0), INVALID), (dict(hq=0), INVALID),
    (dict(hq=8 * 129, qs=1 << 20), INVALID), (dict(d=0), INVALID), (dict(d=257, qs=1 << 20), INVALID),
    (dict(batch=-1), INVALID), (dict(batch=65537), INVALID), (dict(total=-1), INVALID),
    (dict(total=2 ** 30), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(qs=4095), INVALID), (dict(q=None), INVALID),
    (dict(cu=None), INVALID), (dict(out=None), INVALID), (dict(q=ODD), MISALIGNED),
    (dict(out=ODD), MISALIGNED), (dict(lse=ctypes.c_void_p(258)), MISALIGNED),
    (dict(cu=ctypes.c_void_p(258)), MISALIGNED), (dict(ws=None), WORKSPACE),
    (dict(ws=ctypes.c_void_p(264)), WORKSPACE), (dict(bytes=8), WORKSPACE),
    (dict(total=0, q=None, out=None), OK), (dict(batch=0, cu=None), OK),
])
def test_attention_refusals(lib, kw, status):
    assert _tree(lib, **kw) == status
    assert _prompt(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), DTYPE), (dict(ps=0), INVALID), (dict(width=0), INVALID), (dict(pages=0), INVALID),
    (dict(pages=2 ** 28), INVALID), (dict(width=2 ** 27), INVALID), (dict(fmt=1), INVALID),
    (dict(mask=P, words=0), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(kc=None), INVALID), (dict(mask=ctypes.c_void_p(260), words=1), MISALIGNED),
    (dict(table=ctypes.c_void_p(258)), MISALIGNED), (dict(kc=ODD), MISALIGNED),
])
def test_paged_refusals(lib, kw, status):
    assert _tree(lib, **kw) == status


def test_prompt_refuses_overlapping_rows(lib):
    assert _prompt(lib, ks=1023) == INVALID
    assert _prompt(lib, vs=1023) == INVALID
    assert _prompt(lib, k=None) == INVALID
    assert _prompt(lib, v=ODD) == MISALIGNED


def test_workspace_sizes(lib):
    size = lib.dflash2_tree_attention_workspace_size
    assert size(512, 32, 32, 8, 128) >= 2 * 152 * 256 * 130 * 4
    assert size(1, 1, 32, 8, 128) < size(512, 32, 32, 8, 128)
    assert size(512, 32, 30, 8, 128) == 0                    # a shape the call refuses
    assert lib.dflash2_prompt_attention_workspace_size(512, 32, 32, 8, 128) > 0
    assert _tree(lib, bytes=size(32, 2, 32, 8, 128) - 1) == WORKSPACE
