"""Cases of the attention operators: the paged key/value cache (written, quantised as it is
written, read back), the attention of a tree of drafted tokens over it, and the causal attention
of packed prompts.

A verified block needs four steps of one attention layer: the prompts' own attention, the write of
keys and values into the cache, the drafted tokens' attention over that cache, and the read of
cached rows when accepted tokens move or a context is handed on.  Each case is one such call.

Cache layout: keys and values [pages, kv_heads, page_size, head_dim]; slot = page * page_size +
offset; an E4M3 cache holds codes c (uint8) and one exponent byte e per row of head_dim values,
standing for c * 2^(e - 127), with the smallest e in [79, 175] that brings the row's largest
magnitude to at most 448.
"""
import math

import numpy as np
import torch

own = False

# Heads of the shapes that this repository proposes for: hidden 4096 and 5120 with 128 per head,
# eight key/value heads.
_H4096 = {"q_heads": 32, "kv_heads": 8, "head_dim": 128}
_H5120 = {"q_heads": 40, "kv_heads": 8, "head_dim": 128}


def listed():
    kv = {"kv_heads": 8, "head_dim": 128}
    return [
        # one step's drafted blocks (32 requests of 16 positions) go into a bf16 cache
        {"name": "write-block", "op": "write", "cache": "bf16", "dtype": "bf16", "tokens": 512,
         "page": 16, **kv},
        # the prompts of a batch go into an 8-bit cache, and a later chunk reads them back
        {"name": "write-prompt-e4m3", "op": "roundtrip", "cache": "e4m3", "dtype": "bf16",
         "tokens": 20011, "page": 32, **kv},
        # the accepted tokens of a small batch are fetched to be moved to their final slots
        {"name": "read-accepted-e4m3", "op": "read", "cache": "e4m3", "dtype": "f32", "tokens": 77,
         "page": 16, **kv},
        # a long shared context is handed to another instance in bf16
        {"name": "read-context-e4m3", "op": "read", "cache": "e4m3", "dtype": "bf16",
         "tokens": 100003, "page": 64, **kv},
        # the next token of a single request: latency
        {"name": "token-single", "op": "tree", "cache": "bf16", "dtype": "bf16", "batch": 1,
         "draft_min": 1, "draft_max": 1, "ctx_min": 1000, "ctx_max": 1000, "page": 16,
         "tree": False, "lse": False, **_H4096},
        # plain decoding of a ragged batch over an 8-bit cache
        {"name": "token-batch-e4m3", "op": "tree", "cache": "e4m3", "dtype": "bf16", "batch": 64,
         "draft_min": 1, "draft_max": 1, "ctx_min": 0, "ctx_max": 8191, "page": 32, "tree": False,
         "lse": True, **_H4096},
        # verification of drafted blocks of 16 positions, 32 requests
        {"name": "block16", "op": "tree", "cache": "bf16", "dtype": "bf16", "batch": 32,
         "draft_min": 16, "draft_max": 16, "ctx_min": 500, "ctx_max": 8000, "page": 16,
         "tree": False, "lse": False, **_H4096},
        # trees of up to 12 drafted tokens, 128 requests, 8-bit cache, five query heads a group
        {"name": "tree12-e4m3", "op": "tree", "cache": "e4m3", "dtype": "bf16", "batch": 128,
         "draft_min": 1, "draft_max": 12, "ctx_min": 13, "ctx_max": 4096, "page": 16, "tree": True,
         "lse": False, **_H5120},
        # large trees over long contexts, few requests
        {"name": "tree64-long", "op": "tree", "cache": "bf16", "dtype": "bf16", "batch": 4,
         "draft_min": 64, "draft_max": 64, "ctx_min": 30011, "ctx_max": 60000, "page": 64,
         "tree": True, "lse": False, **_H4096},
        # a few short prompts in fp32 (the numerics check of a new checkpoint)
        {"name": "prompt-short-f32", "op": "prompt", "dtype": "f32", "batch": 3, "len_min": 1,
         "len_max": 301, "q_heads": 8, "kv_heads": 2, "head_dim": 64, "lse": True},
        # a packed batch of ordinary prompts
        {"name": "prompt-packed", "op": "prompt", "dtype": "bf16", "batch": 16, "len_min": 100,
         "len_max": 2048, "lse": False, **_H5120},
        # one long document
        {"name": "prompt-long", "op": "prompt", "dtype": "bf16", "batch": 1, "len_min": 12001,
         "len_max": 12001, "lse": False, **_H4096},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "roundtrip", "read", "tree", "tree", "tree", "prompt", "prompt"])
    group = rng.choice([1, 2, 4, 4, 5, 8])
    kv_heads = rng.choice([1, 2, 4, 8, 8])
    head_dim = rng.choice([64, 128, 128])
    cache = rng.choice(["bf16", "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    lse = rng.choice([False, True])
    if op in ("write", "roundtrip", "read"):
        return {"op": op, "cache": "bf16" if op == "write" else cache,
                "dtype": "bf16" if cache == "bf16" or op != "read" else rng.choice(["bf16", "f32"]),
                "tokens": _log_int(rng, 1, 60000), "page": page, "kv_heads": kv_heads,
                "head_dim": head_dim}
    heads = {"q_heads": group * kv_heads, "kv_heads": kv_heads, "head_dim": head_dim}
    if op == "prompt":
        f32 = rng.random() < 0.2
        total = _log_int(rng, 16, 1500 if f32 else 8000)
        batch = rng.randint(1, 12)
        top = max(1, total // batch)
        return {"op": op, "dtype": "f32" if f32 else "bf16", "batch": batch,
                "len_min": rng.randint(1, top), "len_max": top, "lse": lse, **heads}
    batch = _log_int(rng, 1, 160)
    draft = _log_int(rng, 1, 64)
    ctx = _log_int(rng, 16, max(64, min(60000, 240000 // batch)))
    return {"op": op, "cache": cache, "dtype": "bf16", "batch": batch,
            "draft_min": rng.randint(1, draft), "draft_max": draft, "ctx_min": rng.randint(0, ctx),
            "ctx_max": ctx, "page": page, "tree": rng.choice([False, True]), "lse": lse, **heads}


# ---- sizes --------------------------------------------------------------------------------------

def _spread(lo, hi, n):
    """n sizes over [lo, hi], the largest among them, in a mixed order that the case alone fixes."""
    at = (np.arange(1, n + 1) * 0.6180339887498949) % 1.0
    at = (at - at.min()) / max(1e-9, at.max() - at.min()) if n > 1 else np.ones(1)
    return (lo + np.floor(at * (hi - lo) + 0.5)).astype(np.int64)


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _cu(n):
    return np.concatenate([np.zeros(1, np.int64), np.cumsum(n)])


def _tree_sizes(case):
    drafted = _spread(case["draft_min"], case["draft_max"], case["batch"])
    ctx = _spread(case["ctx_min"], case["ctx_max"], case["batch"])[::-1].copy()
    return drafted, ctx


def work(case):
    d, hk = case["head_dim"], case["kv_heads"]
    el = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("write", "roundtrip", "read"):
        rows = 2 * case["tokens"] * hk
        raw, held = rows * d * el, rows * (d * 2 if case["cache"] == "bf16" else d + 1)
        slots = 8 * case["tokens"]
        if case["op"] == "roundtrip":
            return {"bytes": 2 * (raw + held + slots), "flops": 2 * rows * d}
        return {"bytes": raw + held + slots, "flops": rows * d if case["cache"] == "e4m3" else 0}
    hq = case["q_heads"]
    if case["op"] == "prompt":
        lens = _spread(case["len_min"], case["len_max"], case["batch"])
        n = int(lens.sum())
        pairs = int((lens * (lens + 1) // 2).sum())
        return {"bytes": 2 * n * (hq + hk) * d * el + (4 * n * hq if case["lse"] else 0),
                "flops": 4 * d * hq * pairs}
    drafted, ctx = _tree_sizes(case)
    keys = int((drafted + ctx).sum())
    held = d * 2 if case["cache"] == "bf16" else d + 1
    n = int(drafted.sum())
    # a tree's node sees its ancestors and itself, about log2 of the nodes; a chain's half of them
    seen = np.log2(drafted + 1.0) if case["tree"] else (drafted + 1) / 2.0
    return {"bytes": 2 * keys * hk * held + 2 * n * hq * d * el + (4 * n * hq if case["lse"] else 0),
            "flops": int(4 * d * hq * (drafted * (ctx + seen)).sum())}


# ---- inputs -------------------------------------------------------------------------------------

def _randn(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _rows(gen, n, heads, d, dtype):
    """Projected keys or values: unit scale, with channels and tokens of unequal strength."""
    x = torch.randn((n, heads, d), generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn((1, heads, d), generator=gen, device="cuda"))
    x *= torch.exp(0.3 * torch.randn((n, 1, 1), generator=gen, device="cuda"))
    return x.to(dtype)


def _pow2(e):
    """2^e in fp32 for integers e, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _held(x, cache):
    """A cache's contents for rows x [..., head_dim]: (values or codes, exponents or None)."""
    if cache != "e4m3":
        return x.to(_dtype(cache)), None
    x = x.float()
    mant, ex = torch.frexp(x.abs().amax(-1))
    e = torch.where(mant == 0, -48, ex - 9 + (mant > 0.875).int()).clamp(-48, 48)
    codes = (x * _pow2(-e.unsqueeze(-1))).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _value(codes, exps):
    """What a cache's rows stand for, in fp32."""
    if exps is None:
        return codes.float()
    return codes.view(torch.float8_e4m3fn).float() * _pow2(exps.int().unsqueeze(-1) - 127)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, d, hk = _dtype(case["dtype"]), case["head_dim"], case["kv_heads"]
    s = {"case": dict(case), "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] in ("write", "roundtrip", "read"):
        n, ps = case["tokens"], case["page"]
        pages = n // ps + 9
        order = torch.randperm(pages, generator=gen, device="cuda")
        first = int(torch.randint(0, ps, (1,), generator=gen, device="cuda"))
        at = torch.arange(n, device="cuda") + first        # a run of tokens over shuffled pages
        s["slots"] = order[at // ps] * ps + at % ps
        if case["op"] == "read":
            s["k_cache"], s["k_exp"] = _held(_rows(gen, pages * hk * ps, 1, d, torch.bfloat16)
                                             .view(pages, hk, ps, d), case["cache"])
            s["v_cache"], s["v_exp"] = _held(_rows(gen, pages * hk * ps, 1, d, torch.bfloat16)
                                             .view(pages, hk, ps, d), case["cache"])
            return s
        held = torch.uint8 if case["cache"] == "e4m3" else _dtype(case["cache"])
        for nm in ("k", "v"):
            # keys and values as slices of one projection's rows, read in place
            s[nm] = _rows(gen, n, 2 * hk, d, dt)[:, :hk]
            s[nm + "_cache"] = torch.zeros((pages, hk, ps, d), dtype=held, device="cuda")
            s[nm + "_exp"] = (torch.zeros((pages, hk, ps), dtype=torch.uint8, device="cuda")
                              if case["cache"] == "e4m3" else None)
        return s
    hq = case["q_heads"]
    s["scale"] = d ** -0.5
    if case["op"] == "prompt":
        lens = _spread(case["len_min"], case["len_max"], case["batch"])
        n = int(lens.sum())
        s["cu"] = torch.from_numpy(_cu(lens)).to("cuda", torch.int32)
        s["max_len"] = int(lens.max())
        # one packed projection: queries, keys and values of a token side by side
        qkv = _randn(gen, (n, hq + 2 * hk, d), dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        return s
    drafted, ctx = _tree_sizes(case)
    ps, batch, n = case["page"], case["batch"], int(drafted.sum())
    lens = drafted + ctx
    per = -(-lens // ps)
    pages = int(per.sum()) + 3
    order = torch.randperm(pages, generator=gen, device="cuda")
    cols = torch.arange(int(per.max()), device="cuda")[None, :]
    start = torch.from_numpy(_cu(per)[:-1]).cuda()[:, None]
    live = cols < torch.from_numpy(per).cuda()[:, None]
    table = torch.where(live, order[(start + cols).clamp(max=pages - 1)], torch.zeros_like(cols))
    s["page_table"] = table.to(torch.int32).contiguous()
    s["cu"] = torch.from_numpy(_cu(drafted)).to("cuda", torch.int32)
    s["kv_lens"] = torch.from_numpy(lens).to("cuda", torch.int32)
    s["max_draft"], s["max_len"] = int(drafted.max()), int(lens.max())
    s["q"] = _randn(gen, (n, hq, d), dt, 1.5)
    for nm in ("k", "v"):
        held, exps = _held(_randn(gen, (pages, hk, ps, d), torch.bfloat16), case["cache"])
        s[nm + "_cache"], s[nm + "_exp"] = held, exps
    s["mask"] = None
    if case["tree"]:
        # every node's parent is an earlier node, near ones likelier; bit j of a node's word: it
        # sees node j (its ancestors and itself)
        rng = np.random.default_rng(seed)
        t = s["max_draft"]
        seen = np.zeros((batch, t), np.uint64)
        seen[:, 0] = 1
        for j in range(1, t):
            parent = np.maximum(0, j - 1 - np.floor(rng.exponential(max(1, t // 6), batch)).astype(int))
            seen[:, j] = seen[np.arange(batch), parent] | (np.uint64(1) << np.uint64(j))
        packed = seen[np.arange(t)[None, :] < drafted[:, None]]
        s["mask"] = torch.from_numpy(packed.view(np.int64).reshape(n, 1)).cuda()
    return s


# ---- one pass -----------------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from block_draft_proposal_gb300 import dflash2
    case = s["case"]
    if case["op"] == "prompt":
        if "ws" not in s:
            s["ws"] = torch.empty(dflash2.prompt_attention_workspace_size(
                s["q"].shape[0], case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"]),
                dtype=torch.uint8, device="cuda")
        out, lse, _ = dflash2.prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["scale"],
                                               with_lse=case["lse"], workspace=s["ws"],
                                               err=s["err"])
        return (out, lse) if case["lse"] else out
    cache = dflash2.KVCache(s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"])
    if case["op"] == "tree":
        if "ws" not in s:
            s["ws"] = torch.empty(dflash2.tree_attention_workspace_size(
                s["q"].shape[0], case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"]),
                dtype=torch.uint8, device="cuda")
        out, lse, _ = dflash2.tree_attention(s["q"], cache, s["page_table"], s["cu"], s["kv_lens"],
                                             s["scale"], tree_mask=s["mask"], with_lse=case["lse"],
                                             workspace=s["ws"], err=s["err"])
        return (out, lse) if case["lse"] else out
    if case["op"] != "read":
        dflash2.kv_cache_write(cache, s["k"], s["v"], s["slots"], err=s["err"])
        if case["op"] == "write":
            return s["k_cache"], s["v_cache"]
    k, v, _ = dflash2.kv_cache_read(cache, s["slots"], dtype=_dtype(case["dtype"]), err=s["err"])
    return k, v


def _run_plain(s):
    case = s["case"]
    if case["op"] == "prompt":
        return _plain_prompt(s)
    if case["op"] == "tree":
        return _plain_tree(s)
    ps = case["page"]
    page, off = s["slots"] // ps, s["slots"] % ps
    if case["op"] != "read":
        _plain_put(s, "k", page, off)
        _plain_put(s, "v", page, off)
        if case["op"] == "write":
            return s["k_cache"], s["v_cache"]
    return _plain_get(s, "k", page, off), _plain_get(s, "v", page, off)


def _plain_put(s, nm, page, off):
    held, exps = _held(s[nm], s["case"]["cache"])
    s[nm + "_cache"][page, :, off] = held
    if exps is not None:
        s[nm + "_exp"][page, :, off] = exps


def _plain_get(s, nm, page, off):
    exps = s[nm + "_exp"]
    rows = s[nm + "_cache"][page, :, off]
    return _value(rows, None if exps is None else exps[page, :, off]).to(_dtype(s["case"]["dtype"]))


def _attend(q, k, v, hidden, scale):
    """softmax(scale q k^T) v in fp32 over [..., rows, d] x [..., keys, d], where `hidden` marks the
    pairs that do not count; (rows, log of the sum), zero and -inf where nothing counts."""
    z = torch.matmul(q * scale, k.transpose(-1, -2)).masked_fill_(hidden, -math.inf)
    top = z.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / total.clamp(min=1e-30)
    return out, (torch.log(total) + top).squeeze(-1)


def _plain_prompt(s):
    case = s["case"]
    hq, hk, d, n = case["q_heads"], case["kv_heads"], case["head_dim"], s["q"].shape[0]
    g, batch, top = hq // hk, case["batch"], s["max_len"]
    start, size = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    pos = torch.arange(top, device="cuda")
    at = (start[:, None] + pos[None, :]).clamp(max=n - 1)                      # [B, L], padded
    q = s["q"][at].float().view(batch, top, hk, g, d).permute(0, 2, 3, 1, 4)
    k = s["k"][at].float().permute(0, 2, 1, 3)[:, :, None]
    v = s["v"][at].float().permute(0, 2, 1, 3)[:, :, None]
    hidden = pos[None, :] > pos[:, None]
    out, lse = _attend(q, k, v, hidden, s["scale"])
    token = torch.arange(n, device="cuda")
    which = torch.searchsorted(s["cu"][1:].long(), token, right=True)
    where = token - start[which]
    out = out.permute(0, 3, 1, 2, 4)[which, where].reshape(n, hq, d).to(s["q"].dtype)
    if not case["lse"]:
        return out
    return out, lse.permute(0, 3, 1, 2)[which, where].reshape(n, hq)


def _plain_tree(s):
    case = s["case"]
    hq, hk, d, n, ps = (case["q_heads"], case["kv_heads"], case["head_dim"], s["q"].shape[0],
                        case["page"])
    g, batch, t, top = hq // hk, case["batch"], s["max_draft"], s["max_len"]
    start, size = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    node = torch.arange(t, device="cuda")
    at = (start[:, None] + node[None, :]).clamp(max=n - 1)                     # [B, T], padded
    q = s["q"][at].float().view(batch, t, hk, g, d).permute(0, 2, 3, 1, 4)
    q = q.reshape(batch, hk, g * t, d)
    table = s["page_table"].long()
    lines = table.shape[1] * ps

    def rows(nm):
        exps = s[nm + "_exp"]
        x = _value(s[nm + "_cache"][table], None if exps is None else exps[table])
        return x.permute(0, 2, 1, 3, 4).reshape(batch, hk, lines, d)

    # key position l of request b: context below ctx, drafted node l - ctx from there on
    pos = torch.arange(lines, device="cuda")
    ctx = (s["kv_lens"].long() - size)[:, None, None]
    j = pos[None, None, :] - ctx                                               # [B, 1, L]
    if s["mask"] is None:
        sees = j <= node[None, :, None]
    else:
        bits = s["mask"][at][..., 0]                                           # [B, T]
        sees = (j < 0) | ((bits[:, :, None] >> j.clamp(0, 63)) & 1).bool()
    hidden = ~(sees & (j < size[:, None, None]))
    hidden = hidden[:, None, None].expand(batch, 1, g, t, lines).reshape(batch, 1, g * t, lines)
    out, lse = _attend(q, rows("k"), rows("v"), hidden, s["scale"])
    token = torch.arange(n, device="cuda")
    which = torch.searchsorted(s["cu"][1:].long(), token, right=True)
    where = token - start[which]
    out = out.view(batch, hk, g, t, d).permute(0, 3, 1, 2, 4)[which, where]
    out = out.reshape(n, hq, d).to(s["q"].dtype)
    if not case["lse"]:
        return out
    return out, lse.view(batch, hk, g, t).permute(0, 3, 1, 2)[which, where].reshape(n, hq)


# ---- the definition, in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("write", "roundtrip", "read"):
        return _exact_cache(case, s)
    hq, hk, n = case["q_heads"], case["kv_heads"], s["q"].shape[0]
    g = hq // hk
    out = torch.zeros((n, hq, case["head_dim"]), dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    cu = s["cu"].tolist()
    for b in range(case["batch"]):
        t0, t1 = cu[b], cu[b + 1]
        t = t1 - t0
        if t == 0:
            continue
        if case["op"] == "prompt":
            keys, values, length, ctx = s["k"][t0:t1], s["v"][t0:t1], t, 0
        else:
            length = int(s["kv_lens"][b])
            ctx = length - t
            line = torch.arange(length, device="cuda")
            pages = s["page_table"][b].long()[line // case["page"]]
            keys, values = (_exact_rows(s, nm, pages, line % case["page"]) for nm in ("k", "v"))
        allowed = torch.ones((t, length), dtype=torch.bool, device="cuda")
        if s.get("mask") is None:
            allowed = torch.tril(allowed, diagonal=ctx)
        else:
            for j in range(t):
                allowed[:, ctx + j] = ((s["mask"][t0:t1, 0] >> j) & 1) == 1
        for h in range(hq):
            z = s["q"][t0:t1, h].double() @ keys[:, h // g].double().T * case["head_dim"] ** -0.5
            z[~allowed] = -math.inf
            lse[t0:t1, h] = torch.logsumexp(z, -1)
            out[t0:t1, h] = torch.exp(z - lse[t0:t1, h, None]) @ values[:, h // g].double()
            del z
    return (out, lse) if case["lse"] else out


def _power(e):
    """2^e in 64 bits for integers e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_rows(s, nm, pages, offs):
    """The cached rows [len, kv_heads, head_dim] at (page, offset), in 64 bits."""
    x = s[nm + "_cache"][pages, :, offs]
    if s[nm + "_exp"] is None:
        return x.double()
    c = x.long()
    low, field = c & 7, (c >> 3) & 15
    size = torch.where(field == 0, low.double(), 8.0 + low) * _power(field.clamp(min=1) - 10)
    power = _power(s[nm + "_exp"][pages, :, offs].long() - 127)
    return torch.where(c >= 128, -size, size) * power.unsqueeze(-1)


def _exact_cache(case, s):
    page, off = s["slots"] // case["page"], s["slots"] % case["page"]
    if case["op"] == "read":
        return tuple(_exact_rows(s, nm, page, off) for nm in ("k", "v"))
    outs = []
    for nm in ("k", "v"):
        x = s[nm].double()
        if case["cache"] == "e4m3":
            # the nearest E4M3 value, ties to the even significand: steps of 2^(binade - 3)
            amax = x.abs().amax(-1, keepdim=True)
            part, power = torch.frexp(amax / 448)              # ceil(log2(amax / 448))
            e = (power - (part == 0.5).int()).clamp(-48, 48)
            y = x * _power(-e)
            step = _power(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
            x = torch.round(y / step) * step * _power(e)
        if case["op"] == "write":
            whole = torch.zeros(s[nm + "_cache"].shape, dtype=torch.float64, device="cuda")
            whole[page, :, off] = x
            x = whole
        outs.append(x)
    return tuple(outs)
