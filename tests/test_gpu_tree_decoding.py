"""examples/tree_decoding.py: the cache, the prompt's and the trees' attention as a
decoder uses them together."""
import importlib.util
import os

import pytest
import torch

from attention_ref import e4m3_values

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                     "tree_decoding.py")


def _example():
    spec = importlib.util.spec_from_file_location("tree_decoding", _PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _prompts(vocab):
    g = torch.Generator().manual_seed(5)
    return [torch.randint(0, vocab, (n,), generator=g).tolist() for n in (33, 1, 140)]


@pytest.mark.parametrize("dtype,e4m3", [(torch.float32, False), (torch.bfloat16, False),
                                        (torch.bfloat16, True)])
def test_tree_decoding_follows_the_model(dtype, e4m3):
    ex = _example()
    layer = ex.Layer(dtype=dtype)
    prompts = _prompts(layer.vocab)
    out, rounds, seqs = ex.generate(layer, prompts, steps=24, depth=3, width=4, e4m3=e4m3)
    assert int(seqs.err.item()) == 0
    assert all(len(o) >= 24 for o in out)
    assert rounds < 23  # a pass gives a token at least, and the drafts are right now and then

    # every token is the model's choice after the ones before it, up to the arithmetic:
    # the whole sequence through the layer in 64 bits
    tol = {torch.float32: 1e-3, torch.bfloat16: 0.15}[dtype] + (0.35 if e4m3 else 0.0)
    w = {n: getattr(layer, n).double().cpu()
         for n in ("embed", "place", "w_qkv", "w_out", "lm_head")}
    for prompt, tokens in zip(prompts, out):
        ids = torch.tensor(prompt + tokens[:-1])
        x = w["embed"][ids] + w["place"][:len(ids)]
        heads = (x @ w["w_qkv"]).view(len(ids), -1, layer.head_dim)
        g = layer.q_heads // layer.kv_heads
        q, k, v = heads.split([layer.q_heads, layer.kv_heads, layer.kv_heads], dim=1)
        k, v = (t.repeat_interleave(g, dim=1) for t in (k, v))
        z = torch.einsum("thd,nhd->htn", q, k) * layer.scale
        z = z.masked_fill(torch.ones(len(ids), len(ids)).triu(1).bool(), float("-inf"))
        o = torch.einsum("htn,nhd->thd", z.softmax(-1), v).reshape(len(ids), -1)
        logits = (x + o @ w["w_out"]) @ w["lm_head"].T
        logits = logits[len(prompt) - 1:]
        chosen = logits.gather(1, torch.tensor(tokens)[:, None])[:, 0]
        assert float((logits.amax(-1) - chosen).max()) <= tol


@pytest.mark.parametrize("e4m3", [False, True])
def test_accepted_rows_lie_where_the_sequence_continues(e4m3):
    ex = _example()
    layer = ex.Layer(dtype=torch.bfloat16)
    prompts = _prompts(layer.vocab)
    out, _, seqs = ex.generate(layer, prompts, steps=16, depth=3, width=4, e4m3=e4m3)
    for b, (prompt, tokens) in enumerate(zip(prompts, out)):
        ids = (prompt + tokens)[:seqs.lens[b]]
        assert seqs.lens[b] == len(prompt) + len(tokens) - 1
        slots = torch.tensor(seqs.slots(b, range(len(ids))))
        pages, line = slots // seqs.page_size, slots % seqs.page_size
        # keys are a function of token and position, up to the projection's rounding
        # (a library product, whose sums may differ with the number of rows)
        x = layer.embed[torch.tensor(ids).cuda()] + layer.place[:len(ids)]
        heads = (x.double() @ layer.w_qkv.double()).view(len(ids), -1, layer.head_dim).cpu()
        k, v = heads[:, layer.q_heads:].split([layer.kv_heads] * 2, dim=1)
        for got, exps, want in ((seqs.cache.k, seqs.cache.k_exp, k), (seqs.cache.v, seqs.cache.v_exp, v)):
            rows = got.cpu()[pages, :, line]
            if e4m3:
                scale = 2.0 ** (exps.cpu()[pages, :, line].double() - 127)
                rows = e4m3_values()[rows.long()] * scale[..., None]
                # a code step is at most 2^-3 of the value, 2^-9 of the row's largest below
                step = want.abs() * 2.0 ** -3 + want.abs().amax(-1, keepdim=True) * 2.0 ** -8
            else:
                step = want.abs() * 2.0 ** -7 + 2.0 ** -12
            assert bool(((rows.double() - want).abs() <= step).all())
