"""What the binding of the cache and attention operators refuses before it calls the library."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from block_draft_proposal_gb300 import dflash2


class _Library:
    """Accepts every call; sizes are 64 bytes."""

    def __getattr__(self, name):
        return lambda *args: 64 if "size" in name else dflash2.OK


@pytest.fixture(autouse=True)
def accepting(monkeypatch):
    monkeypatch.setattr(dflash2, "library", _Library)
    monkeypatch.setattr(dflash2, "_ptr", lambda t: None if t is None else 256)
    monkeypatch.setattr(dflash2, "_stream", lambda s: 0)
    with FakeTensorMode():
        yield


def _t(*shape, dtype=torch.bfloat16, device="cuda"):
    return torch.zeros(shape, dtype=dtype, device=device)


def _tree(**kw):
    return dflash2.tree_attention(_t(3, 4, 64), dflash2.new_kv_cache(4, 16, 2, 64), _t(2, 2, dtype=torch.int32),
                                  _t(3, dtype=torch.int32), _t(2, dtype=torch.int32), 0.1, **kw)


def test_a_mask_without_words():
    _tree(tree_mask=_t(3, 1, dtype=torch.int64))
    with pytest.raises(ValueError):                     # it would be taken for a chain
        _tree(tree_mask=_t(3, 0, dtype=torch.int64))
    with pytest.raises(ValueError):
        _tree(tree_mask=_t(3, dtype=torch.int64))


def _write(**kw):
    return dflash2.kv_cache_write(dflash2.new_kv_cache(4, 16, 2, 64), _t(3, 2, 64), _t(3, 2, 64),
                                  _t(3, dtype=torch.int64), **kw)


def _read(**kw):
    return dflash2.kv_cache_read(dflash2.new_kv_cache(4, 16, 2, 64), _t(3, dtype=torch.int64), **kw)


def _prompt(**kw):
    return dflash2.prompt_attention(_t(3, 4, 64), _t(3, 2, 64), _t(3, 2, 64), _t(3, dtype=torch.int32), 0.1, **kw)


@pytest.mark.parametrize("call", [_write, _read, _tree, _prompt])
def test_error_words(call):
    call(err=_t(1, dtype=torch.int32))
    call(err=_t(4, dtype=torch.int32))
    for bad, kind in ((_t(1, dtype=torch.int32, device="cpu"), ValueError), (_t(1, dtype=torch.int64), TypeError),
                      (_t(0, dtype=torch.int32), ValueError)):
        with pytest.raises(kind):
            call(err=bad)


@pytest.mark.parametrize("call", [_tree, _prompt])
def test_workspaces(call):
    call(workspace=_t(64, dtype=torch.uint8))
    for bad in (_t(64, dtype=torch.uint8, device="cpu"), _t(128, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            call(workspace=bad)
