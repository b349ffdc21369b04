"""The norms, the E4M3 block products and the rotary positions reject bad arguments on the host,
before any CUDA call.  No compute call is made."""
import ctypes

import pytest

P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(257)
OK, INVALID, DTYPE, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build_library()
    from block_draft_proposal_gb300 import dflash2
    return dflash2.library()


def _quantise(lib, **kw):
    a = dict(x=P, stride=300, rows=4, cols=300, dtype=1, q=P, scale=P)
    a.update(kw)
    return lib.dflash2_quantize_blocks_e4m3(a["x"], a["stride"], a["rows"], a["cols"], a["dtype"], a["q"], a["scale"],
                                            None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), DTYPE), (dict(rows=-1), INVALID), (dict(rows=2 ** 31), INVALID), (dict(cols=0), INVALID),
    (dict(stride=299), INVALID), (dict(stride=2 ** 33), INVALID), (dict(x=None), INVALID), (dict(q=None), INVALID),
    (dict(scale=None), INVALID), (dict(x=ODD), MISALIGNED), (dict(scale=ctypes.c_void_p(258)), MISALIGNED),
    (dict(rows=2 ** 31 - 1, cols=2 ** 31 - 1, stride=2 ** 31), INVALID), (dict(rows=0, x=None), OK),
])
def test_quantise_refusals(lib, kw, status):
    assert _quantise(lib, **kw) == status


def _linear(lib, **kw):
    a = dict(x=P, stride=256, xt=1, xq=None, xs=None, w=P, ws=P, rows=4, n_in=256, n_out=130, ot=1, out=P, work=P,
             bytes=1 << 40, err=P)
    a.update(kw)
    return lib.dflash2_linear_fp8_blocks(a["x"], a["stride"], a["xt"], a["xq"], a["xs"], a["w"], a["ws"], a["rows"],
                                         a["n_in"], a["n_out"], a["ot"], a["out"], a["work"], a["bytes"], a["err"],
                                         None)


@pytest.mark.parametrize("kw,status", [
    (dict(xt=2), DTYPE), (dict(ot=-1), DTYPE), (dict(rows=-1), INVALID), (dict(rows=2 ** 20 + 1), INVALID),
    (dict(n_in=0, stride=0), INVALID), (dict(n_out=0), INVALID), (dict(n_out=2 ** 24, n_in=2 ** 17, stride=2 ** 17), INVALID),
    (dict(rows=2 ** 18, n_out=2 ** 22, n_in=16, stride=16), INVALID), (dict(stride=255), INVALID), (dict(n_in=248), MISALIGNED), (dict(x=None), INVALID), (dict(xq=P, xs=P), INVALID),
    (dict(x=None, xq=P), INVALID), (dict(w=None), INVALID), (dict(ws=None), INVALID), (dict(out=None), INVALID),
    (dict(x=ODD), MISALIGNED), (dict(w=ctypes.c_void_p(264)), MISALIGNED), (dict(out=ODD), MISALIGNED),
    (dict(ws=ctypes.c_void_p(258)), MISALIGNED), (dict(err=ODD), MISALIGNED),
    (dict(x=None, xq=ctypes.c_void_p(264), xs=P), MISALIGNED), (dict(work=None), WORKSPACE),
    (dict(work=ctypes.c_void_p(264)), WORKSPACE), (dict(bytes=64), WORKSPACE),
    (dict(rows=0, x=None, out=None), OK), (dict(rows=0, x=None, xq=None, work=None), OK),
])
def test_linear_refusals(lib, kw, status):
    assert _linear(lib, **kw) == status


def test_linear_workspace(lib):
    size = lib.dflash2_linear_fp8_blocks_workspace_size
    assert size(5, 272, 1000) >= 5 * 272 + 5 * 3 * 4
    assert size(-1, 272, 1000) == 0 and size(5, 0, 10) == 0
    assert _linear(lib, bytes=size(4, 256, 130) - 1) == WORKSPACE


def _norm(lib, **kw):
    a = dict(x=P, stride=300, xt=0, w=P, offset=1.0, eps=1e-6, rows=4, hidden=300, dtype=1, out=P, scale=None)
    a.update(kw)
    return lib.dflash2_sublayer_norm(a["x"], a["stride"], a["xt"], a["w"], a["offset"], a["eps"], a["rows"],
                                     a["hidden"], a["dtype"], a["out"], a["scale"], None)


def _join(lib, **kw):
    a = dict(x=P, stride=300, xt=0, y=P, ys=300, post=P, gate=P, kind=3, gs=300, act=1, branch=0.5, w=P, offset=1.0,
             eps=1e-6, rows=4, hidden=300, dtype=1, ro=ctypes.c_void_p(1 << 20), ros=300, out=P, scale=None)
    a.update(kw)
    return lib.dflash2_sublayer_join(a["x"], a["stride"], a["xt"], a["y"], a["ys"], a["post"], a["gate"], a["kind"],
                                     a["gs"], a["act"], a["branch"], a["w"], a["offset"], a["eps"], a["rows"],
                                     a["hidden"], a["dtype"], a["ro"], a["ros"], a["out"], a["scale"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(xt=2), DTYPE), (dict(dtype=5), DTYPE), (dict(rows=-1), INVALID), (dict(rows=2 ** 31), INVALID),
    (dict(hidden=0), INVALID), (dict(hidden=32769, stride=32769), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(offset=NAN), INVALID), (dict(stride=299), INVALID),
    (dict(stride=2 ** 33), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(x=ODD), MISALIGNED),
    (dict(w=ODD), MISALIGNED), (dict(out=ODD), MISALIGNED), (dict(out=ODD, scale=ctypes.c_void_p(258)), MISALIGNED),
    (dict(rows=0, x=None, out=None, w=None), OK),
])
def test_norm_refusals(lib, kw, status):
    assert _norm(lib, **kw) == status
    assert _join(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(kind=4), INVALID), (dict(kind=-1), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID),
    (dict(branch=INF), INVALID), (dict(ys=299), INVALID), (dict(gs=299), INVALID), (dict(kind=2, gs=0), INVALID),
    (dict(ros=299), INVALID), (dict(y=None), INVALID), (dict(ro=None), INVALID), (dict(gate=None), INVALID),
    (dict(w=None), INVALID), (dict(w=None, out=None, scale=P), INVALID), (dict(ro=P, ros=304), INVALID),
    (dict(y=ODD), MISALIGNED), (dict(gate=ODD), MISALIGNED), (dict(post=ODD), MISALIGNED), (dict(ro=ODD), MISALIGNED),
])
def test_join_refusals(lib, kw, status):
    assert _join(lib, **kw) == status


def test_norm_needs_its_weight(lib):
    assert _norm(lib, w=None) == INVALID


BASE = dict(q=P, qs=2048, k=P, ks=512, v=P, vs=512, pos=P, axes=3, freq=P, axis=P, rot=64, adj=0, mag=1.0, slots=P, n=4,
            hq=16, hk=4, d=128, ps=16, pages=10, dtype=1, fmt=0, qo=ctypes.c_void_p(1 << 20), qos=2048, ko=ctypes.c_void_p(1 << 21),
            kos=512, kc=P, vc=P, ke=None, ve=None, err=P)


def _rotary(lib, **kw):
    a = {**BASE, **kw}
    return lib.dflash2_rotary(a["q"], a["qs"], a["k"], a["ks"], a["pos"], a["axes"], a["freq"], a["axis"], a["rot"],
                              a["adj"], a["mag"], a["n"], a["hq"], a["hk"], a["d"], a["dtype"], a["qo"], a["qos"],
                              a["ko"], a["kos"], a["err"], None)


def _rotary_write(lib, **kw):
    a = {**BASE, **kw}
    return lib.dflash2_rotary_kv_write(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["axes"],
                                       a["freq"], a["axis"], a["rot"], a["adj"], a["mag"], a["slots"], a["n"], a["hq"],
                                       a["hk"], a["d"], a["ps"], a["pages"], a["dtype"], a["fmt"], a["qo"], a["qos"],
                                       a["ko"], a["kos"], a["kc"], a["vc"], a["ke"], a["ve"], a["err"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), DTYPE), (dict(d=0, rot=0), INVALID), (dict(d=257), INVALID), (dict(rot=0), INVALID),
    (dict(rot=63), INVALID), (dict(rot=130), INVALID), (dict(axes=0), INVALID), (dict(axes=256), INVALID),
    (dict(adj=2), INVALID), (dict(mag=NAN), INVALID), (dict(n=-1), INVALID), (dict(hq=-1), INVALID),
    (dict(hk=-1), INVALID), (dict(n=2 ** 31), INVALID), (dict(n=2 ** 28), INVALID), (dict(qs=2047), INVALID),
    (dict(hq=2 ** 17, qs=2 ** 24, qos=2 ** 24), INVALID), (dict(qos=2047), INVALID), (dict(ks=511), INVALID),
    (dict(kos=511), INVALID), (dict(qs=2 ** 33), INVALID), (dict(pos=None), INVALID), (dict(freq=None), INVALID),
    (dict(axis=None), INVALID), (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(k=None), INVALID),
    (dict(qo=P, qos=4096), INVALID), (dict(ko=P, kos=1024), INVALID), (dict(q=ODD), MISALIGNED), (dict(k=ODD), MISALIGNED),
    (dict(qo=ODD), MISALIGNED), (dict(ko=ODD), MISALIGNED), (dict(pos=ctypes.c_void_p(260)), MISALIGNED),
    (dict(freq=ctypes.c_void_p(260)), MISALIGNED), (dict(err=ODD), MISALIGNED), (dict(n=0, q=None, k=None), OK),
])
def test_rotary_refusals(lib, kw, status):
    assert _rotary(lib, **kw) == status
    assert _rotary_write(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), DTYPE), (dict(hk=0), INVALID), (dict(ps=0), INVALID), (dict(pages=-1), INVALID),
    (dict(pages=2 ** 60), INVALID), (dict(vs=511), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID),
    (dict(kc=None), INVALID), (dict(fmt=1), INVALID), (dict(fmt=1, ke=P), INVALID), (dict(v=ODD), MISALIGNED),
    (dict(vc=ODD), MISALIGNED), (dict(slots=ctypes.c_void_p(260)), MISALIGNED),
])
def test_rotary_write_refusals(lib, kw, status):
    assert _rotary_write(lib, **kw) == status


def test_rotary_needs_something_to_turn(lib):
    assert _rotary(lib, hq=0, hk=0) == INVALID
    assert _rotary(lib, ko=None) == INVALID
