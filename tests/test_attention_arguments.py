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
