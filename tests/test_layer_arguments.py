"""What the binding of the norms, block products and rotary positions refuses before it calls the
library, and that what a call allocates belongs to its stream."""
import contextlib

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from block_draft_proposal_gb300 import dflash2


class _Library:
    """Accepts every call; sizes are 64 bytes."""

    def __getattr__(self, name):
        return lambda *args: 64 if "size" in name else dflash2.OK


class _Stream:
    cuda_stream = 7


@pytest.fixture(autouse=True)
def allocations(monkeypatch):
    """(name, the stream it was allocated in or None) of every allocation."""
    now, log = [], []

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    for name in ("empty", "zeros", "full", "empty_like", "zeros_like"):
        def alloc(*a, _make=getattr(torch, name), _name=name, **k):
            log.append((_name, now[-1] if now else None))
            return _make(*a, **k)
        monkeypatch.setattr(torch, name, alloc)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(dflash2, "library", _Library)
    monkeypatch.setattr(dflash2, "_ptr", lambda t: None if t is None else 256)
    monkeypatch.setattr(dflash2, "_stream", lambda s: 0 if s is None else s.cuda_stream)
    monkeypatch.setattr(dflash2, "_current_device", lambda: 0)
    monkeypatch.setattr(dflash2, "_one_device", False)
    with FakeTensorMode():
        yield log


def _t(*shape, dtype=torch.bfloat16, device="cuda"):
    return torch.randn(shape, device=device).to(dtype)


def _i(*shape, dtype=torch.int64, device="cuda"):
    return torch.ones(shape, dtype=dtype, device=device)


U8, F32 = torch.uint8, torch.float32


def _norm(x=None, w=None, **kw):
    return dflash2.sublayer_norm(_t(3, 256) if x is None else x, _t(256) if w is None else w, **kw)


def _join(x=None, y=None, **kw):
    return dflash2.sublayer_join(_t(3, 256) if x is None else x, _t(3, 256) if y is None else y,
                                 **{"next_weight": _t(256), **kw})


def _linear(x=None, w=None, s=None, **kw):
    return dflash2.linear_fp8_blocks(_t(3, 256) if x is None else x, _i(130, 256, dtype=U8) if w is None else w,
                                     _t(2, 2, dtype=F32) if s is None else s, **kw)


def _table(half=32):
    return dflash2.RotaryTable(_i(half), _i(half, dtype=U8))


def _rotary(q=None, k=None, pos=None, table=None, **kw):
    return dflash2.rotary(_t(3, 4, 64) if q is None else q, _t(3, 2, 64) if k is None else k,
                          _i(3) if pos is None else pos, table or _table(), **kw)


def _write(q=None, k=None, v=None, slots=None, **kw):
    return dflash2.rotary_kv_write(dflash2.new_kv_cache(4, 16, 2, 64), _t(3, 4, 64) if q is None else q,
                                   _t(3, 2, 64) if k is None else k, _t(3, 2, 64) if v is None else v, _i(3, 3),
                                   _table(), _i(3) if slots is None else slots, **kw)


def _quantise(**kw):
    return dflash2.quantize_blocks_e4m3(_t(3, 256), **kw)


@pytest.mark.parametrize("call", [_quantise, _norm, _join, lambda **k: _join(e4m3=True, **k), _linear, _rotary, _write,
                                  lambda **k: _write(with_k=True, **k)])
def test_a_call_allocates_in_its_stream(allocations, call, monkeypatch):
    marks = []
    check = dflash2._check
    real = {n: getattr(dflash2, n) for n in ("quantize_blocks_e4m3", "sublayer_norm", "sublayer_join",
                                             "linear_fp8_blocks", "rotary", "rotary_kv_write")}
    for name, fn in real.items():
        def marked(*a, _fn=fn, **k):
            marks.append(len(allocations))
            return _fn(*a, **k)
        monkeypatch.setattr(dflash2, name, marked)
    for stream in (None, _Stream()):
        call(stream=stream)
        made = allocations[marks[-1]:]
        assert made and all(s is stream for _, s in made), made
    assert check is dflash2._check


def test_outputs_and_their_types():
    out, scale = _norm(_t(3, 256, dtype=F32))
    assert out.dtype == torch.bfloat16 and scale is None
    out, scale = _norm(e4m3=True)
    assert out.dtype == U8 and scale.shape == (3, 2) and scale.dtype == F32
    r, out, scale = _join(_t(3, 256, dtype=F32))
    assert r.dtype == F32 and out.dtype == torch.bfloat16 and scale is None
    assert _join(next_weight=None)[1:] == (None, None)
    assert _linear()[0].dtype == torch.bfloat16 and _linear(_t(3, 256, dtype=F32))[0].dtype == F32
    codes = _linear(_i(3, 256, dtype=U8), x_scale=_t(3, 2, dtype=F32))
    assert codes[0].dtype == torch.bfloat16 and codes[0].shape == (3, 130)
    assert _linear(out_dtype=F32)[0].dtype == F32
    assert _linear(out=_t(3, 130, dtype=F32))[0].dtype == F32
    assert _write()[1] is None and _write(with_k=True)[1].shape == (3, 2, 64)
    _norm(_t(3, 512)[:, :256])
    _join(_t(3, 512)[:, :256], _t(3, 512)[:, 256:], gate=_t(3, 256))
    _join(gate=_t(256))
    _join(gate=_t(3, 1))
    _rotary(pos=_i(2, 3))
    _rotary(q=_t(3, 8, 64)[:, :4])


@pytest.mark.parametrize("call", [
    lambda: _norm(_t(3, 256, device="cpu")), lambda: _norm(_t(256)), lambda: _norm(_t(256, 3).T),
    lambda: _norm(_t(1, 256).expand(3, 256)), lambda: _norm(w=_t(255)), lambda: _norm(out=_t(3, 255)),
    lambda: _norm(scale=_t(3, 2, dtype=F32)), lambda: _norm(e4m3=True, scale=_t(3, 3, dtype=F32)),
    lambda: _join(y=_t(3, 255)), lambda: _join(gate=_t(255)), lambda: _join(gate=_t(2, 256)),
    lambda: _join(gate=_t(3, 2)), lambda: _join(gate=_t()), lambda: _join(gate_act="relu"), lambda: _join(post_weight=_t(128)),
    lambda: _join(next_weight=None, e4m3=True), lambda: _join(next_weight=None, out=_t(3, 256)),
    lambda: _join(residual_out=_t(2, 256)), lambda: _join(residual_out=_t(1, 256).expand(3, 256)),
    lambda: _linear(_t(3, 255)), lambda: _linear(s=_t(2, 3, dtype=F32)), lambda: _linear(_i(3, 256, dtype=U8)),
    lambda: _linear(x_scale=_t(3, 2, dtype=F32)), lambda: _linear(_i(3, 256, dtype=U8), x_scale=_t(3, 1, dtype=F32)),
    lambda: _linear(out=_t(3, 131)), lambda: _linear(workspace=_i(64, dtype=U8, device="cpu")),
    lambda: _linear(err=_i(1, dtype=torch.int32, device="cpu")), lambda: _linear(_i(3, 512, dtype=U8)[:, :256], x_scale=_t(3, 2, dtype=F32)),
    lambda: _rotary(pos=_i(4)), lambda: _rotary(pos=_i(3, 2)), lambda: _rotary(k=_t(2, 2, 64)),
    lambda: _rotary(k=_t(3, 2, 32)), lambda: _rotary(k=_t(3, 2, 64, dtype=F32)), lambda: _rotary(q_out=_t(3, 2, 64)),
    lambda: _rotary(table=dflash2.RotaryTable(_i(32), _i(31, dtype=U8))), lambda: _rotary(q=_t(3, 64, 4).transpose(1, 2)),
    lambda: dflash2.rotary(_t(3, 4, 64), None, _i(3), _table(), k_out=_t(3, 2, 64)),
    lambda: _write(slots=_i(2)), lambda: _write(v=_t(3, 1, 64)), lambda: _write(q=_t(2, 4, 64)),
    lambda: _write(k=_t(3, 4, 64)), lambda: _write(q=_t(3, 4, 64, dtype=F32)),
    lambda: _quantise(q=_i(3, 255, dtype=U8)), lambda: _quantise(scale=_t(3, 1, dtype=F32)),
])
def test_shapes_and_places(call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("call", [
    lambda: _norm(_i(3, 256)), lambda: _norm(w=_i(256)), lambda: _norm(out=_t(3, 256, dtype=F32)),
    lambda: _norm(e4m3=True, out=_t(3, 256)), lambda: _join(gate=_t(256, dtype=F32)),
    lambda: _join(post_weight=_t(256, dtype=F32)), lambda: _join(residual_out=_t(3, 256, dtype=F32)),
    lambda: _linear(_t(3, 256, dtype=torch.float16)), lambda: _linear(w=_i(130, 256)), lambda: _linear(s=_t(2, 2)),
    lambda: _linear(out_dtype=F32, out=_t(3, 130)), lambda: _rotary(pos=_i(3, dtype=torch.int32)),
    lambda: _rotary(table=dflash2.RotaryTable(_t(32), _i(32, dtype=U8))),
    lambda: _rotary(table=dflash2.RotaryTable(_i(32), _i(32))), lambda: _write(slots=_i(3, dtype=torch.int32)),
    lambda: _write(v=_t(3, 2, 64, dtype=F32)),
])
def test_types(call):
    with pytest.raises(TypeError):
        call()


@pytest.mark.parametrize("kw", [dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, sections=[1, 2]),
                                dict(rotary_dim=8, inv_freq=[1.0]), dict(rotary_dim=8, sections=[-1, 5]),
                                dict(rotary_dim=8, sections=[1, 3], interleaved=True)])
def test_tables(kw):
    with pytest.raises(ValueError):
        dflash2.rotary_table(**kw)


@pytest.mark.parametrize("call", [_quantise, _norm, _join, _linear, _rotary, _write])
def test_another_device_than_the_current_one(call, monkeypatch):
    call()
    monkeypatch.setattr(dflash2, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        call()


def test_tensors_of_two_devices():
    there = "cuda:1"
    for call in (lambda: _norm(w=_t(256, device=there)), lambda: _join(gate=_t(256, device=there)),
                 lambda: _linear(s=_t(2, 2, dtype=F32, device=there)), lambda: _rotary(pos=_i(3, device=there)),
                 lambda: _write(slots=_i(3, device=there)),
                 lambda: _rotary(table=dflash2.RotaryTable(_i(32, device=there), _i(32, dtype=U8, device=there)))):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_a_cache_of_two_devices():
    there = "cuda:1"
    n, heads, d = 3, 2, 64
    kv, exps = (4, heads, 16, d), (4, heads, 16)
    for cache in (dflash2.KVCache(_t(*kv), _t(*kv, device=there)),
                  dflash2.KVCache(_i(*kv, dtype=U8), _i(*kv, dtype=U8), _i(*exps, dtype=U8, device=there), _i(*exps, dtype=U8)),
                  dflash2.KVCache(_i(*kv, dtype=U8), _i(*kv, dtype=U8), _i(*exps, dtype=U8), _i(*exps, dtype=U8, device=there))):
        with pytest.raises(ValueError, match="current device"):
            dflash2.rotary_kv_write(cache, None, _t(n, heads, d), _t(n, heads, d), _i(n), _table(), _i(n))
