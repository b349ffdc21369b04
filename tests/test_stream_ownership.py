"""What a call with `stream` allocates belongs to that stream: torch's allocator hands the memory
of a dropped tensor to later work of the stream it was allocated in, so that a workspace of the
current stream could be overwritten while the call still uses it."""
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


@pytest.fixture
def seen(monkeypatch):
    """(name, the stream it was allocated in or None) of every allocation of a call."""
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
    with FakeTensorMode():
        yield log


def _t(*shape, dtype=torch.bfloat16):
    return torch.randn(shape, device="cuda").to(dtype)


def _i(*shape, dtype=torch.int32):
    return torch.ones(shape, dtype=dtype, device="cuda")


def _cache(e4m3=False):
    return dflash2.new_kv_cache(4, 16, 2, 64, e4m3=e4m3)


def _walk():
    return dict(anchor_ids=_i(2, dtype=torch.int64), cand_ids=_i(2, 3, 4, dtype=torch.int64),
                cand_u=_t(2, 3, 4, dtype=torch.float32), temperatures=_t(2, dtype=torch.float32),
                greedy=_i(2, dtype=torch.uint8), uniforms=_t(2, 3, dtype=torch.float32),
                with_path_scores=True)


I64, F32 = torch.int64, torch.float32
CALLS = {
    "kv_cache_write": lambda s: dflash2.kv_cache_write(_cache(), _t(3, 2, 64), _t(3, 2, 64), _i(3, dtype=I64),
                                                       stream=s),
    "kv_cache_read": lambda s: dflash2.kv_cache_read(_cache(True), _i(3, dtype=I64), stream=s),
    "tree_attention": lambda s: dflash2.tree_attention(_t(3, 4, 64), _cache(), _i(2, 2), _i(3), _i(2), 0.1,
                                                       with_lse=True, stream=s),
    "prompt_attention": lambda s: dflash2.prompt_attention(_t(3, 4, 64), _t(3, 2, 64), _t(3, 2, 64), _i(3), 0.1,
                                                           with_lse=True, stream=s),
    "grouped_conv": lambda s: dflash2.grouped_conv(_t(4, 64), _t(3, 64), _t(4, 3 * 4), 4, 16, 3, stream=s),
    "conv_prepare": lambda s: dflash2.conv_prepare(_t(4, 64), _t(2 * 3 * 4, 64), _t(2, 3, 64), 4, 16, 3, stream=s),
    "conv_finish": lambda s: dflash2.conv_finish(_t(4, 64), _t(4, 2, 3, 4), _t(2, 3, 64), 4, 16, 3, stream=s),
    "unary_topk": lambda s: dflash2.unary_topk(_t(4, 64), _t(32, 64), 32, 1.0, 0.0, 4, stream=s),
    "unary_topk_fp8": lambda s: dflash2.unary_topk_fp8(_t(4, 64), _i(32, 64, dtype=torch.uint8), _t(32, dtype=F32),
                                                       32, 1.0, 0.0, 4, stream=s),
    "quantize_rows_e4m3": lambda s: dflash2.quantize_rows_e4m3(_t(4, 64), stream=s),
    "quantize_rows_nvfp4": lambda s: dflash2.quantize_rows_nvfp4(_t(4, 64), stream=s),
    "nvfp4_tile_scales": lambda s: dflash2.nvfp4_tile_scales(_i(4, 4, dtype=torch.uint8), 64, stream=s),
    "unary_topk_nvfp4": lambda s: dflash2.unary_topk_nvfp4(_t(4, 64), _i(32, 32, dtype=torch.uint8),
                                                           _i(64, dtype=torch.uint8), 1.0, 32, 1.0, 0.0, 4,
                                                           stream=s),
    "topk_merge": lambda s: dflash2.topk_merge(_i(2, 3, 4, dtype=I64), _t(2, 3, 4, dtype=F32), (0, 8), 4, stream=s),
    "selector_walk": lambda s: dflash2.selector_walk(_t(6, 64), _t(8, 64), _t(32, 8), _t(32, 8), **_walk(), stream=s),
    "selector_walk_projected": lambda s: dflash2.selector_walk_projected(
        _t(32, 8), _t(32, 8), hidden=64, workspace=_i(64, dtype=torch.uint8), **_walk(), stream=s),
    "selector_walk_noalloc": lambda s: dflash2.selector_walk_noalloc(_t(6, 64), _t(8, 64), _t(32, 8), _t(32, 8),
                                                                     **_walk(), stream=s),
    "d2t_remap": lambda s: dflash2.d2t_remap(_i(4, dtype=I64), None, 32, 32, stream=s),
    "verify": lambda s: dflash2.verify(_t(2, 4, 32), _t(2, dtype=F32), _i(2, dtype=torch.uint8), _i(2, 3, dtype=I64),
                                       _i(2, 3, 4, dtype=I64), _t(2, 3, 4, dtype=F32), _t(2, 4, dtype=F32), stream=s),
    "philox_uniforms": lambda s: dflash2.philox_uniforms(1, 8, device="cuda", stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_call_allocates_in_its_stream(seen, name, monkeypatch):
    real, marks = getattr(dflash2, name), []

    def call(*a, **k):  # the inputs are made before
        marks.append(len(seen))
        return real(*a, **k)

    monkeypatch.setattr(dflash2, name, call)
    for stream in (None, _Stream()):
        CALLS[name](stream)
        made = seen[marks[-1]:]
        assert made and all(s is stream for _, s in made), made


@pytest.mark.gpu
def test_a_workspace_is_not_handed_on_while_it_is_used(cuda):
    from test_gpu_attention import Case
    c = Case([16] * 5 + [40], [900, 10, 3000, 129, 64, 5000], 16, 4, 128, 32, seed=41)
    args = (c.q, c.cache, c.table.cuda(), c.cu.cuda(), c.lens.cuda(), c.scale)
    want, lse, _ = c.run()
    size = dflash2.tree_attention_workspace_size(sum(c.t), 6, 16, 4, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                     # some 10 ms: the call starts behind it
    out, lse2, err = dflash2.tree_attention(*args, with_lse=True, stream=side)
    mine = [torch.full((size,), 0x5A, dtype=torch.uint8, device=cuda) for _ in range(3)]
    side.synchronize()
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(out, want) and torch.equal(lse, lse2)
    assert all(bool((m == 0x5A).all()) for m in mine)
