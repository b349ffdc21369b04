"""Decoding with drafted trees over a paged cache: the prompt's attention, the
cache write, the attention of each drafted tree, and the accepted rows' move.

    python examples/tree_decoding.py [--e4m3] [--float32]

The model is one attention layer with random weights over random embeddings, so
that the program is about the calls, not about the text.  Each round drafts a tree
of candidates (unary_topk), runs the whole tree through the layer in one pass,
follows the model's own choices down the tree as far as it was drafted, and moves
the accepted nodes' keys and values to where the sequences continue.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from block_draft_proposal_gb300 import dflash2  # noqa: E402


class Layer:
    """Embedding, one layer of grouped-query attention, and the output head."""

    def __init__(self, vocab=512, hidden=512, q_heads=8, kv_heads=2, head_dim=64,
                 dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rows = (q_heads + 2 * kv_heads) * head_dim

        def w(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(device, dtype)

        self.vocab, self.q_heads, self.kv_heads, self.head_dim = vocab, q_heads, kv_heads, head_dim
        self.dtype, self.device = dtype, torch.device(device)
        self.scale = 1.0 / math.sqrt(head_dim)
        self.embed = w(vocab, hidden, std=1.0)
        self.place = w(4096, hidden, std=0.5)
        self.w_qkv = w(hidden, rows, std=1.0 / math.sqrt(hidden))
        self.w_out = w(q_heads * head_dim, hidden, std=1.0 / math.sqrt(q_heads * head_dim))
        self.lm_head = w(vocab, hidden, std=1.0 / math.sqrt(hidden))

    def project(self, tokens, positions):
        """(x, q, k, v) of packed tokens; q, k and v are slices of one projection."""
        x = self.embed[tokens] + self.place[positions]
        heads = (x @ self.w_qkv).view(-1, self.q_heads + 2 * self.kv_heads, self.head_dim)
        return (x, *heads.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1))

    def hidden(self, x, attended):
        return x + attended.reshape(len(x), -1) @ self.w_out

    def logits(self, h):
        return (h @ self.lm_head.T).float()


class Sequences:
    """A batch of sequences in a paged cache; `room` positions each."""

    def __init__(self, layer, batch, room, page_size=16, e4m3=False):
        self.layer, self.batch, self.page_size = layer, batch, page_size
        per = -(-room // page_size)
        self.cache = dflash2.new_kv_cache(batch * per, page_size, layer.kv_heads, layer.head_dim,
                                          layer.dtype, e4m3, layer.device)
        # the requests' pages lie interleaved, as they would after some serving
        self.table = torch.arange(batch * per, dtype=torch.int32).view(per, batch).T.contiguous()
        self.pages = self.table.to(layer.device)
        self.lens = [0] * batch
        self.err = torch.zeros(1, dtype=torch.int32, device=layer.device)

    def slots(self, b, positions):
        return [int(self.table[b, i // self.page_size]) * self.page_size + i % self.page_size
                for i in positions]

    def on_device(self, values, dtype):
        return torch.tensor(values, dtype=dtype, device=self.layer.device)

    def prefill(self, prompts):
        """Packed prompts through the layer and into the cache; each one's last
        hidden state."""
        layer = self.layer
        cu = [0]
        slots, positions = [], []
        for b, prompt in enumerate(prompts):
            cu.append(cu[-1] + len(prompt))
            slots += self.slots(b, range(len(prompt)))
            positions += range(len(prompt))
            self.lens[b] = len(prompt)
        tokens = self.on_device([t for prompt in prompts for t in prompt], torch.int64)
        x, q, k, v = layer.project(tokens, self.on_device(positions, torch.int64))
        out, _, _ = dflash2.prompt_attention(q, k, v, self.on_device(cu, torch.int32), layer.scale,
                                             err=self.err)
        dflash2.kv_cache_write(self.cache, k, v, self.on_device(slots, torch.int64), err=self.err)
        return layer.hidden(x, out)[self.on_device(cu[1:], torch.int64) - 1]

    def tree_pass(self, trees):
        """trees[b] = (tokens, parents) with parents[i] < i, or -1 for the root: the
        nodes' hidden states, per request.  Their rows lie behind the sequence."""
        layer = self.layer
        cu, slots, positions, tokens, words = [0], [], [], [], []
        for b, (toks, parents) in enumerate(trees):
            depth, seen = [], []
            for i, parent in enumerate(parents):
                depth.append(0 if parent < 0 else depth[parent] + 1)
                seen.append((1 << i) | (0 if parent < 0 else seen[parent]))
            cu.append(cu[-1] + len(toks))
            tokens += toks
            positions += [self.lens[b] + d for d in depth]
            slots += self.slots(b, range(self.lens[b], self.lens[b] + len(toks)))
            words += [[s - (1 << 64) if s >> 63 else s] for s in seen]
        x, q, k, v = layer.project(self.on_device(tokens, torch.int64),
                                   self.on_device(positions, torch.int64))
        dflash2.kv_cache_write(self.cache, k, v, self.on_device(slots, torch.int64), err=self.err)
        lens = [n + len(t[0]) for n, t in zip(self.lens, trees)]
        out, _, _ = dflash2.tree_attention(
            q, self.cache, self.pages, self.on_device(cu, torch.int32),
            self.on_device(lens, torch.int32), layer.scale,
            tree_mask=self.on_device(words, torch.int64), err=self.err)
        return layer.hidden(x, out).split([len(t[0]) for t in trees])

    def keep(self, paths):
        """paths[b]: the accepted nodes, root first.  Their rows move to the
        sequence's next positions.  All are read before any is written, and a
        row that is read back from codes and written again keeps its values."""
        src, dst = [], []
        for b, path in enumerate(paths):
            for i, node in enumerate(path):
                if node != i:
                    src += self.slots(b, [self.lens[b] + node])
                    dst += self.slots(b, [self.lens[b] + i])
            self.lens[b] += len(path)
        if src:
            k, v, _ = dflash2.kv_cache_read(self.cache, self.on_device(src, torch.int64),
                                            dtype=self.layer.dtype, err=self.err)
            dflash2.kv_cache_write(self.cache, k, v, self.on_device(dst, torch.int64), err=self.err)


def draft(layer, seqs, last, depth, width):
    """A tree per request: the sampled token `last`, then `depth` levels of the
    `width` best candidates after the best node of the level before.  The drafter is
    the model without its attention: the output head on the token's embedding."""
    trees = [([token], [-1]) for token in last]
    at = [0] * len(last)
    for level in range(depth):
        h = layer.embed[seqs.on_device([t[0][i] for t, i in zip(trees, at)], torch.int64)]
        h = h + layer.place[seqs.on_device([n + level for n in seqs.lens], torch.int64)]
        ids, _, _ = dflash2.unary_topk(h, layer.lm_head, layer.vocab, 1.0, 0.0, width, err=seqs.err)
        for b, row in enumerate(ids.tolist()):
            tokens, parents = trees[b]
            parents += [at[b]] * width
            at[b] = len(tokens)
            tokens += row
    return trees


def generate(layer, prompts, steps, depth=3, width=4, e4m3=False):
    """At least `steps` greedy tokens per prompt: (tokens, rounds, sequences).
    depth 0 drafts nothing: a token per pass."""
    seqs = Sequences(layer, len(prompts), max(map(len, prompts)) + steps + 2 * (1 + depth * width),
                     e4m3=e4m3)
    out = [[t] for t in layer.logits(seqs.prefill(prompts)).argmax(-1).tolist()]
    rounds = 0
    while min(map(len, out)) < steps:
        last = [o[-1] for o in out]
        # a finished sequence has an empty tree
        trees = draft(layer, seqs, last, depth, width)
        trees = [t if len(o) < steps else ([], []) for t, o in zip(trees, out)]
        hidden = seqs.tree_pass(trees)
        paths = []
        for b, ((tokens, parents), hb) in enumerate(zip(trees, hidden)):
            path = []
            if tokens:
                best = layer.logits(hb).argmax(-1).tolist()
                node = 0
                while node is not None:
                    path.append(node)
                    out[b].append(best[node])
                    node = next((i for i in range(node + 1, len(tokens))
                                 if parents[i] == node and tokens[i] == best[node]), None)
            paths.append(path)
        seqs.keep(paths)
        rounds += 1
    return out, rounds, seqs


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--e4m3", action="store_true", help="hold the cache as E4M3 codes")
    ap.add_argument("--float32", action="store_true")
    a = ap.parse_args()
    layer = Layer(dtype=torch.float32 if a.float32 else torch.bfloat16)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, layer.vocab, (n,), generator=g).tolist() for n in (37, 5, 130, 1)]
    out, rounds, seqs = generate(layer, prompts, steps=32, e4m3=a.e4m3)
    if int(seqs.err.item()):
        raise SystemExit(f"device error word {int(seqs.err.item())}")
    for prompt, tokens in zip(prompts, out):
        print(f"prompt of {len(prompt):3d}: {len(tokens)} tokens, {tokens[:8]} ...")
    print(f"{rounds} passes, {sum(map(len, out)) / len(out) / rounds:.2f} tokens per pass")


if __name__ == "__main__":
    main()
