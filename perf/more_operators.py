"""Decoding drafted tokens over a paged cache, as measured cases: the operators that a step with a draft
model (or draft heads) makes, and the windows with sinks that keep a long conversation's cache small.

    gqa_tree_mask        positions and visibility bits of trees of drafted tokens, from their parents
    gqa_paged_append     with a norm of each query and key head before the rotation, at given positions
    nvfp4_paged_append   the same into NVFP4 pages
    gqa_paged_tree_attn  attention of several new tokens per sequence, a tree or a chain, over a paged cache
    gqa_paged_attn       of one new token with a sliding window and a few first tokens that stay visible
    gqa_paged_keep       the accepted tokens' cache rows moved together, the others' given up

With ``own`` false, run() computes the plain form in elementary torch operations; with ``own`` true it
makes the library calls.  exact() is the definition in 64 bits.
"""
import math

import torch

own = False
DEV = "cuda"

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZES = {"f16": 2, "bf16": 2, "e4m3": 1}
ROPE_BASE = 500000.0
EPS = 1e-6
K_SCALE, V_SCALE = 0.0625, 0.03125  # E4M3 pages: stored value = value / scale
Q_SCALE = 0.03125                   # NVFP4 path: E4M3 query = query / scale


# ------------------------------------------------------------------ cases ---

def _append(name, type, cache, batch, q_len, kv_len, hq, hkv, d, rot, page, layout, interleaved, ragged, tree):
    c = dict(op="append", type=type, cache=cache, batch=batch, q_len=q_len, kv_len=kv_len, hq=hq, hkv=hkv, d=d, rot=rot,
             page=page, layout=layout, interleaved=interleaved, ragged=ragged, tree=tree)
    return dict(name=name, **c) if name else c


def _sinks(name, type, cache, batch, kv_len, hq, hkv, d, page, layout, window, sinks, softcap, ragged):
    c = dict(op="sinks", type=type, cache=cache, batch=batch, q_len=1, kv_len=kv_len, hq=hq, hkv=hkv, d=d, page=page,
             layout=layout, window=window, sinks=sinks, softcap=softcap, ragged=ragged, tree=False)
    return dict(name=name, **c) if name else c


def _tree(name, type, cache, batch, q_len, kv_len, hq, hkv, d, page, layout, window, sinks, softcap, ragged, tree):
    c = dict(op="tree", type=type, cache=cache, batch=batch, q_len=q_len, kv_len=kv_len, hq=hq, hkv=hkv, d=d, page=page,
             layout=layout, window=window, sinks=sinks, softcap=softcap, ragged=ragged, tree=tree)
    return dict(name=name, **c) if name else c


def _mask(name, batch, q_len, kv_len, window, sinks, ragged):
    c = dict(op="mask", batch=batch, q_len=q_len, kv_len=kv_len, window=window, sinks=sinks, ragged=ragged, tree=True)
    return dict(name=name, **c) if name else c


def _keep(name, type, layers, batch, q_len, kv_len, accept, hkv, d, page, layout, ragged):
    c = dict(op="keep", type=type, layers=layers, batch=batch, q_len=q_len, kv_len=kv_len, accept=accept, hkv=hkv, d=d,
             page=page, layout=layout, ragged=ragged, tree=True)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one conversation, a tree of 16 drafted tokens: once for all layers of a step
        _mask("mask_b1_n16", 1, 16, 1024, 0, 0, False),
        # a full serving batch with trees of up to 64, in a model with a window
        _mask("mask_b256_n64", 256, 64, 2048, 16, 4, True),
        # one sequence, one new token, heads normed: a chat turn's decode step, where the launch is what counts
        _append("norm_append_b1", "bf16", "bf16", 1, 1, 1024, 32, 8, 128, 128, 64, "hnd", False, False, False),
        # prompts: batch 4 of 2048 tokens
        _append("norm_append_b4_q2048", "bf16", "bf16", 4, 2048, 2048, 32, 8, 128, 128, 64, "hnd", False, False, False),
        # one conversation far beyond its window
        _sinks("sinks_b1_kv32768", "bf16", "bf16", 1, 32768, 32, 8, 128, 64, "hnd", 4096, 4, 0.0, False),
        # a serving batch of ragged lengths up to 16001 in E4M3 pages, windows of 4096 behind 4 sinks
        _sinks("sinks_b48_e4m3", "bf16", "e4m3", 48, 16001, 64, 8, 128, 16, "nhd", 4096, 4, 0.0, True),
        # one conversation, a small tree: verification of 8 drafted tokens
        _tree("tree_b1_n8_kv2048", "bf16", "bf16", 1, 8, 2048, 32, 8, 128, 64, "hnd", 0, 0, 0.0, False, True),
        # chains of 5 drafted tokens, window, sinks and capped scores, head dim 256, two query heads per KV head
        _tree("chain_b33_n5_window", "bf16", "bf16", 33, 5, 6007, 16, 8, 256, 32, "nhd", 4096, 16, 50.0, True, False),
        # a serving batch with trees of up to 16, eight query heads per KV head over an E4M3 cache
        _tree("tree_b48_n16_e4m3", "bf16", "e4m3", 48, 16, 16001, 64, 8, 128, 16, "nhd", 0, 0, 0.0, True, True),
        # long contexts with trees of 64 tokens: 256 rows a KV head
        _tree("tree_b8_n64_kv65536", "f16", "f16", 8, 64, 65536, 32, 8, 128, 64, "hnd", 0, 0, 0.0, False, True),
        # one conversation's accepted tokens, one layer
        _keep("keep_b1", "bf16", 1, 1, 16, 1024, 4, 8, 128, 64, "hnd", False),
        # a serving batch's, in the pages of 16 layers
        _keep("keep_b64_layers16", "bf16", 16, 64, 64, 200, 8, 8, 128, 16, "hnd", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = [(32, 8), (64, 8), (16, 8), (8, 8), (28, 4), (16, 1), (5, 1), (40, 2), (12, 12)]
    page, layout = rng.choice([16, 32, 64, 128]), rng.choice(["hnd", "nhd"])
    kind = rng.choice(["append", "append", "nvfp4", "sinks", "sinks", "tree", "tree", "tree", "tree", "mask", "keep"])
    window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 16, 4096), rng.choice([0, 1, 4, 100]))])
    if kind == "mask":
        return _mask(None, _log(rng, 1, 400), _log(rng, 1, 150), 150 + _log(rng, 1, 4000), rng.choice([0, 3, 16]), sinks,
                     rng.random() < 0.6)
    if kind == "nvfp4":
        batch = _log(rng, 1, 24)
        q_len = _log(rng, 1, 8192 // batch)
        kv_len = q_len + rng.choice([0, rng.randint(0, 200)])
        return _append(None, rng.choice(["f16", "bf16"]), "nvfp4", batch, q_len, kv_len, 32, 8, 128, rng.choice([128, 128, 64]), 64,
                       "hnd", rng.random() < 0.3, batch > 1 and rng.random() < 0.6, q_len <= 64 and rng.random() < 0.5)
    type = rng.choice(["f16", "bf16"])
    cache = rng.choice([type, type, "e4m3"])
    hq, hkv = rng.choice(heads)
    d = rng.choice([64, 128, 128, 256])
    if kind == "keep":
        layers, batch, q_len = _log(rng, 1, 32), _log(rng, 1, 128), _log(rng, 2, 64)
        room = 400_000_000 // (2 * hkv * d * 2 * layers * batch)
        return _keep(None, cache, layers, batch, q_len, q_len + _log(rng, 1, max(2, min(2000, room))), _log(rng, 1, 9), hkv, d, page,
                     layout, batch > 1 and rng.random() < 0.6)
    if kind == "append":
        room = min(16384, 200_000_000 // ((hq + 2 * hkv) * d * 2))
        batch = _log(rng, 1, min(256, room))
        q_len = rng.choice([1, _log(rng, 1, max(1, room // batch))])
        kv_len = q_len + _log(rng, 1, 400) - 1
        return _append(None, type, cache, batch, q_len, kv_len, hq, hkv, d, rng.choice([r for r in (32, 64, 128, 256) if r <= d]),
                       page, layout, rng.random() < 0.4, batch > 1 and rng.random() < 0.6, q_len <= 64 and rng.random() < 0.5)
    cap = rng.choice([0.0, 0.0, 30.0])
    if kind == "sinks":
        room = 4_000_000_000 // (2 * hkv * d * 2)
        batch = _log(rng, 1, 256)
        kv_len = _log(rng, 1, max(2, min(131072, room // batch)))
        return _sinks(None, type, cache, batch, kv_len, hq, hkv, d, page, layout, _log(rng, 16, 4096), rng.choice([1, 4, 4, 100, 1000]),
                      cap, batch > 1 and rng.random() < 0.7)
    batch, q_len = _log(rng, 1, 64), _log(rng, 1, rng.choice([8, 16, 64, 64, 100]))
    room = min(2_000_000_000 // (2 * hkv * d * 2), 1_000_000_000 // (hq * q_len), 120_000_000_000 // (hq * q_len * d))
    kv_len = q_len + _log(rng, 1, max(2, min(131072, room // batch)))
    return _tree(None, type, cache, batch, q_len, kv_len, hq, hkv, d, page, layout, window, sinks, cap,
                 batch > 1 and rng.random() < 0.7, rng.random() < 0.75)


def _spread(n, b, ragged):
    """All n, or evenly spread from 1 to n."""
    return [n] * b if not ragged or b == 1 else [1 + (n - 1) * i // (b - 1) for i in range(b)]


def _lengths(case):
    """(new tokens, cached ones before them) of each sequence."""
    b, n = case["batch"], case["q_len"]
    new = _spread(n, b, case["ragged"])
    if case["op"] == "append":  # the same number of cached tokens before each chunk
        return new, [case["kv_len"] - n] * b
    return new[::-1], [x - 1 for x in _spread(case["kv_len"] - n + 1, b, case["ragged"])]


def _accepted(case):
    """How many of a sequence's drafted tokens were accepted: none for every fifth sequence of a batch."""
    new, _ = _lengths(case)
    return [0 if i % 5 == 4 else min(1 + (7 * i + case["accept"] - 1) % case["accept"], n - 1) for i, n in enumerate(new)]


# ----------------------------------------------------------------- inputs ---

def _pages(gen, dtype, num, hkv, page, d, layout, layers=0):
    """[(layers,) num, hkv, page, d] (a view where the storage is token-major), filled as an older cache is."""
    n = num * max(1, layers)
    shape = (n, page, hkv, d) if layout == "nhd" else (n, hkv, page, d)
    t = torch.empty(shape, dtype=dtype, device=DEV)
    for i in range(0, n, 4096):
        x = torch.empty((min(4096, n - i),) + shape[1:], dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
        t[i:i + 4096] = (x * 16).clamp(-448, 448).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)
    t = t.permute(0, 2, 1, 3) if layout == "nhd" else t
    return t.unflatten(0, (layers, num)) if layers else t


def _table(gen, kv_lens, page):
    """Block table [batch, max pages] of shuffled physical pages; -1 behind a sequence's last page."""
    n = [(x + page - 1) // page for x in kv_lens]
    perm = torch.randperm(max(1, sum(n)), generator=gen, device=DEV).to(torch.int32)
    used = torch.arange(max(1, max(n)), device=DEV)[None, :] < torch.tensor(n, device=DEV)[:, None]
    table = torch.full(used.shape, -1, dtype=torch.int32, device=DEV)
    table[used] = perm[:sum(n)]
    return table, max(1, sum(n))


def _rope_table(length, rot):
    inv = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    angle = torch.arange(length, dtype=torch.float64, device=DEV)[:, None] * inv[None, :]
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def _parents(gen, index):
    """A random parent before each token of a tree: the last cached token (-1), or a drafted one."""
    u = torch.rand(index.shape, generator=gen, device=DEV, dtype=torch.float64)
    return (u * (index + 1).double()).long().sub(1).minimum(index - 1).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    b = case["batch"]
    order = torch.randperm(b, generator=gen, device=DEV).tolist()
    new, before = _lengths(case)
    new, before = [new[i] for i in order], [before[i] for i in order]
    lens = [x + y for x, y in zip(new, before)]
    s = dict(case=case)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["indptr"] = torch.tensor([0] + new, dtype=torch.int32, device=DEV).cumsum(0).to(torch.int32)
    s["seq"] = torch.repeat_interleave(torch.arange(b, device=DEV), torch.tensor(new, device=DEV))
    index = torch.arange(sum(new), device=DEV) - s["indptr"][s["seq"]]
    if case["tree"] and case["op"] != "keep":
        s["parents"] = _parents(gen, index)
    if case["op"] == "mask":
        return s
    hkv, d, page = case["hkv"], case["d"], case["page"]
    s["table"], num = _table(gen, lens, page)
    if case["op"] == "keep":
        # a path's tokens in order; the one that stands first was not the accepted one, so that each row moves
        count = [_accepted(case)[i] for i in order]
        kept = torch.full((b, max(1, max(count))), -1, dtype=torch.int32, device=DEV)
        for i, (n, m) in enumerate(zip(new, count)):
            kept[i, :m] = torch.randperm(max(1, n - 1), generator=gen, device=DEV)[:m].sort().values.to(torch.int32) + 1
        s["kept"], s["count"] = kept, torch.tensor(count, dtype=torch.int32, device=DEV)
        for name in ("k", "v"):
            s[name] = _pages(gen, DTYPES[case["type"]], num, hkv, page, d, case["layout"], case["layers"])
        return s
    hq, dtype = case["hq"], DTYPES[case["type"]]
    if case["tree"]:
        # (an earlier part of the step has made them)
        window, sinks = (case["window"], case["sinks"]) if case["op"] == "tree" else (0, 0)
        s["mask"], s["positions"] = _tree_plain(s, window, sinks)
    if case["op"] == "append":
        # q, k and v as a fused projection leaves them: slices of one row per token
        qkv = torch.empty(sum(new), hq + 2 * hkv, d, dtype=dtype, device=DEV).normal_(generator=gen)
        qkv[:, hq:hq + hkv, ::16] *= 4  # keys have channels that stand out
        s["q"], s["k_new"], s["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_norm"], s["k_norm"] = torch.rand(2, d, generator=gen, device=DEV).mul(2).add(0.25).to(dtype)
        s["rope"] = _rope_table(max(lens), case["rot"])
    else:
        s["q"] = (torch.empty(sum(new), hq, d, device=DEV).normal_(generator=gen) * 1.5).to(dtype)
    if case["cache"] == "nvfp4":
        # codes [K|V, pages, heads, tokens, d / 2] and scales [K|V, pages, heads, tokens, d / 16]
        s["codes"] = torch.randint(0, 256, (2, num, hkv, page, d // 2), generator=gen, device=DEV, dtype=torch.uint8)
        s["sf"] = torch.rand(2, num, hkv, page, d // 16, generator=gen, device=DEV).add(0.1).to(torch.float8_e4m3fn)
        mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
        vals = torch.cat([mags, -mags]).half()
        byte = torch.arange(256, device=DEV)
        s["values"] = torch.stack([vals[byte % 16], vals[byte // 16]], dim=1)  # the two values of a byte
        return s
    s["k"] = _pages(gen, DTYPES[case["cache"]], num, hkv, page, d, case["layout"])
    s["v"] = _pages(gen, DTYPES[case["cache"]], num, hkv, page, d, case["layout"])
    s["scales"] = (K_SCALE, V_SCALE) if case["cache"] == "e4m3" else (1.0, 1.0)
    return s


# ------------------------------------------------------------------- run ----

def run(state):
    case = state["case"]
    if case["op"] == "mask":
        mask, positions = _mask_own(state) if own else _tree_plain(state, case["window"], case["sinks"])
        return {"mask": mask, "positions": positions}
    if case["op"] == "keep":
        lens = _keep_own(state) if own else _keep_plain(state)
        return {"k": state["k"], "v": state["v"], "lens": lens}
    if case["op"] == "sinks":
        return _sinks_own(state) if own else _attn_plain(state)
    if case["op"] == "tree":
        return _tree_own(state) if own else _attn_plain(state)
    if case["cache"] == "nvfp4":
        q = _nvfp4_own(state) if own else _nvfp4_plain(state)
        # the codes as the values that they stand for
        values = torch.nn.functional.embedding(state["codes"].int(), state["values"])
        return {"q": q, "values": values, "sf": state["sf"]}
    q = _append_own(state) if own else _append_plain(state)
    return {"q": q, "k": state["k"], "v": state["v"]}


def _mask_own(s):
    import gqa_attention_kv_split_gb300 as gqa
    case = s["case"]
    return gqa.gqa_tree_mask(s["parents"], s["indptr"], s["lens"], max_tokens=case["q_len"], window=case["window"], sinks=case["sinks"])


def _keep_own(s):
    import gqa_attention_kv_split_gb300 as gqa
    return gqa.gqa_paged_keep((s["k"], s["v"]), s["table"], s["indptr"], s["lens"], s["kept"], s["count"])


def _append_own(s):
    import gqa_attention_kv_split_gb300 as gqa
    case = s["case"]
    return gqa.gqa_paged_append(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"],
                                qo_indptr=None if case["q_len"] == 1 else s["indptr"], rope=s["rope"],
                                interleaved=case["interleaved"], k_scale=s["scales"][0], v_scale=s["scales"][1],
                                positions=s["positions"] if case["tree"] else None, q_norm=s["q_norm"], k_norm=s["k_norm"],
                                norm_eps=EPS)


def _nvfp4_own(s):
    import gqa_attention_kv_split_gb300 as gqa
    case = s["case"]
    q = gqa.nvfp4_paged_append(s["q"], s["k_new"], s["v_new"], s["codes"][0], s["sf"][0], s["codes"][1], s["sf"][1], s["table"],
                               s["indptr"], s["lens"], rope=s["rope"], interleaved=case["interleaved"], q_scale=Q_SCALE,
                               positions=s["positions"] if case["tree"] else None, q_norm=s["q_norm"], k_norm=s["k_norm"], norm_eps=EPS)
    return q.view(torch.float8_e4m3fn)


def _sinks_own(s):
    import gqa_attention_kv_split_gb300 as gqa
    case = s["case"]
    lse = torch.empty(case["batch"], case["hq"], dtype=torch.float32, device=s["q"].device)
    out = gqa.gqa_paged_attn(s["q"], s["k"], s["v"], s["table"], s["lens"], lse=lse, window=case["window"], sinks=case["sinks"],
                             softcap=case["softcap"], k_scale=s["scales"][0], v_scale=s["scales"][1])
    return {"out": out, "lse": lse}


def _tree_own(s):
    import gqa_attention_kv_split_gb300 as gqa
    case = s["case"]
    lse = torch.empty(s["q"].shape[0], case["hq"], dtype=torch.float32, device=s["q"].device)
    out = gqa.gqa_paged_tree_attn(s["q"], s["k"], s["v"], s["table"], s["indptr"], s["lens"], mask=s.get("mask"),
                                  positions=s.get("positions"), lse=lse, window=case["window"], sinks=case["sinks"],
                                  softcap=case["softcap"], k_scale=s["scales"][0], v_scale=s["scales"][1])
    return {"out": out, "lse": lse}


def _index(s):
    """Each token's number among its sequence's new ones."""
    return torch.arange(s["seq"].shape[0], device=DEV) - s["indptr"][s["seq"]]


def _closed(reach, n):
    """The reflexive relation [b, n, n] and what it leads to: squared until a path of n steps is in it."""
    return reach if n <= 1 else _closed(torch.matmul(reach, reach).clamp(max=1), (n + 1) // 2)


def _tree_plain(s, window, sinks):
    """Bits of the tokens of its tree that a token sees (itself and those above it), and its position."""
    n, b = s["case"]["q_len"], s["case"]["batch"]
    i, seq, at = _index(s), s["seq"], torch.arange(n, device=DEV)
    reach = torch.eye(n, device=DEV).repeat(b, 1, 1)
    above = s["parents"].long()
    reach[seq[above >= 0], i[above >= 0], above[above >= 0]] = 1
    reach = _closed(reach, n) > 0                                              # [b, n, n]: j is i or above it
    depth = reach.sum(-1) - 1                                                  # (of a token that is not there: 0)
    before = s["lens"] - (s["indptr"][1:] - s["indptr"][:-1])
    if window:
        far = (depth[:, None, :] + window <= depth[:, :, None]) & (before[:, None] + depth >= sinks)[:, None, :]
        reach = reach & ~far
    words = (n + 31) // 32
    bits = torch.nn.functional.pad(reach, (0, 32 * words - n)).unflatten(-1, (words, 32)).long()
    packed = (bits << torch.arange(32, device=DEV)).sum(-1)
    packed = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(torch.int32)
    return packed[seq, i], (before[seq] + depth[seq, i]).to(torch.int32)


def _keep_plain(s):
    new = s["indptr"][1:] - s["indptr"][:-1]
    before, page = s["lens"] - new, s["case"]["page"]
    at = torch.arange(s["kept"].shape[1], device=DEV)
    seq, j = torch.nonzero(at[None, :] < s["count"][:, None], as_tuple=True)
    src, dst = before[seq] + s["kept"][seq, j], before[seq] + j
    src_page, dst_page = s["table"][seq, src // page].long(), s["table"][seq, dst // page].long()
    _moved(s["k"], src_page, src % page, dst_page, dst % page)
    _moved(s["v"], src_page, src % page, dst_page, dst % page)
    return before + s["count"]


def _moved(pages, src_page, src, dst_page, dst):
    x = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
    x = x.permute(1, 3, 0, 2, 4)  # [page, slot, layer, head, d]
    x[dst_page, dst] = x[src_page, src]


def _places(s):
    """Position, page and slot of each new token."""
    pos = _index(s) - (s["indptr"][1:] - s["indptr"][:-1])[s["seq"]] + s["lens"][s["seq"]]
    page = s["case"]["page"]
    return pos, s["table"][s["seq"], pos // page].long(), pos % page


def _normed(x, weight):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _rotate(x, cos, sin, interleaved):
    """Rotary embedding of the first 2 * cos.shape[-1] elements of each head."""
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., 2 * half:]], dim=-1)


def _turned(s, pos):
    """q and k normed and rotated to their positions, and v, in 32 bits."""
    half = s["case"]["rot"] // 2
    cs = s["rope"][s["positions"].long() if s["case"]["tree"] else pos]
    cos, sin, inter = cs[:, :half], cs[:, half:], s["case"]["interleaved"]
    return (_rotate(_normed(s["q"], s["q_norm"]), cos, sin, inter), _rotate(_normed(s["k_new"], s["k_norm"]), cos, sin, inter),
            s["v_new"].float())


def _rounded(x, dtype, scale):
    """x / scale in `dtype`; E4M3 saturates."""
    if scale != 1.0:
        x = x * torch.tensor(1.0 / scale, dtype=torch.float32, device=x.device)
    return x.clamp(-448, 448).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)


def _append_plain(s):
    pos, page, slot = _places(s)
    q, k, v = _turned(s, pos)
    _placed(s["k"], page, slot, _rounded(k, s["k"].dtype, s["scales"][0]))
    _placed(s["v"], page, slot, _rounded(v, s["v"].dtype, s["scales"][1]))
    return q.to(s["q"].dtype)


def _placed(pages, page, slot, y):
    if pages.dtype == torch.float8_e4m3fn:
        pages, y = pages.view(torch.uint8), y.view(torch.uint8)
    pages[page, :, slot] = y


def _nvfp4_plain(s):
    pos, page, slot = _places(s)
    q, k, v = _turned(s, pos)
    six = torch.tensor(6.0, device=DEV)
    x = torch.stack([k, v]).unflatten(-1, (-1, 16))                        # [2, T, heads, blocks, 16]
    sf = (x.abs().amax(-1) / six).clamp(max=448).to(torch.float8_e4m3fn)
    scale = sf.float()[..., None]
    y = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0)
    a = y.abs()
    # nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code: whether a tie goes up alternates
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5).byte() + 8 * torch.signbit(y).byte())
    code = code.flatten(-2)
    packed = code[..., 0::2] + 16 * code[..., 1::2]
    s["codes"][:, page, :, slot] = packed.transpose(0, 1)
    s["sf"].view(torch.uint8)[:, page, :, slot] = sf.view(torch.uint8).transpose(0, 1)
    return _rounded(q, torch.float8_e4m3fn, Q_SCALE)


def _gathered(pages, table):
    """The pages of each sequence in order: [batch, heads, tokens, d] in 32 bits."""
    raw = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
    x = raw[table.clamp(min=0).long()]
    if pages.dtype == torch.float8_e4m3fn:
        x = x.view(torch.float8_e4m3fn)
    return x.permute(0, 2, 1, 3, 4).float().flatten(2, 3)


def _seen(s, t):
    """Which of the tokens t of a sequence each of its new ones sees: [batch, q_len, tokens]."""
    case = s["case"]
    n = (s["indptr"][1:] - s["indptr"][:-1])[:, None, None]
    i = torch.arange(case["q_len"], device=DEV)[None, :, None]
    lens, t = s["lens"][:, None, None], t[None, None, :]
    base = lens - n
    at = base + i                                                          # its place in the cache
    if not case["tree"]:
        seen = t <= at
        if case["window"]:
            seen = seen & ((t > at - case["window"]) | (t < case["sinks"]))
        return seen & (i < n)
    row = (s["indptr"][:-1, None] + i[..., 0]).clamp(max=s["seq"].shape[0] - 1)  # [batch, q_len]
    cached = t < base
    if case["window"]:
        cached = cached & ((t > s["positions"][row][..., None] - case["window"]) | (t < case["sinks"]))
    bits = ((s["mask"][row][..., None] >> torch.arange(32, device=DEV)) & 1).flatten(-2) > 0     # [batch, q_len, 32 words]
    drafted = torch.gather(bits, 2, (t - base).clamp(0, bits.shape[2] - 1).expand(-1, case["q_len"], -1))
    return (cached | ((t >= base) & (t < lens) & drafted)) & (i < n)


def _attn_plain(s):
    case = s["case"]
    b, hq, hkv, d, n = case["batch"], case["hq"], case["hkv"], case["d"], case["q_len"]
    i = _index(s)
    q = torch.zeros(b, n, hq, d, device=DEV)
    q[s["seq"], i] = s["q"].float()
    q = q.view(b, n, hkv, hq // hkv, d).transpose(1, 2).flatten(2, 3)      # [b, hkv, n * group, d]
    k = _gathered(s["k"], s["table"])
    x = torch.matmul(q, k.transpose(-1, -2)) * (s["scales"][0] / math.sqrt(d))
    del k
    if case["softcap"]:
        x = torch.tanh(x / case["softcap"]) * case["softcap"]
    t = torch.arange(x.shape[-1], device=DEV)
    seen = _seen(s, t)[:, None, :, None, :]                                # [b, 1, n, 1, tokens]
    x = torch.where(seen, x.view(b, hkv, n, hq // hkv, -1), -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.where(seen, torch.exp(x - m), 0.0)
    total = x.sum(-1, keepdim=True)
    v = torch.where((t[None, :] < s["lens"][:, None])[:, None, :, None], _gathered(s["v"], s["table"]), 0.0)
    out = torch.matmul(x.flatten(2, 3), v).view(b, hkv, n, hq // hkv, d)
    out = torch.where(total > 0, out / total * s["scales"][1], 0.0).transpose(1, 2).flatten(2, 3)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)[..., 0].transpose(1, 2).flatten(2, 3)
    return {"out": out[s["seq"], i].to(s["q"].dtype), "lse": lse[s["seq"], i]}


# ------------------------------------------------------------------- work ---

def work(case):
    new, before = _lengths(case)
    b, total = case["batch"], sum(new)
    if case["op"] == "mask":
        words = (case["q_len"] + 31) // 32
        return {"bytes": 4 * (total * (2 + words) + 2 * b + 1), "flops": total * words}
    hkv, d, page = case["hkv"], case["d"], case["page"]
    if case["op"] == "keep":
        rows = sum(_accepted(case))
        return {"bytes": 2 * rows * case["layers"] * 2 * hkv * d * SIZES[case["type"]] + 4 * (rows + 4 * b), "flops": 0}
    hq, w = case["hq"], SIZES[case["type"]]
    if case["op"] != "append":
        window, sinks = case["window"], case["sinks"]
        read = pairs = pages = 0
        for n, c in zip(new, before):
            first = min(max(0, c + 1 - window) if window else 0, c)  # of the first new token's window
            seen = c - first + min(sinks, first)
            read += seen + n
            pages += (seen + n + page - 1) // page
            pairs += n * seen + (n * (n + 1) // 2 if not case["tree"] else n * max(1, n.bit_length()))
        return {"bytes": 2 * read * hkv * d * SIZES[case["cache"]] + 2 * total * hq * d * w + 4 * total * hq + 4 * pages + 8 * b,
                "flops": 4 * pairs * hq * d}
    out = w * hq
    if case["cache"] == "nvfp4":
        stored = 2 * hkv * d * (0.5 + 1 / 16)
        out = hq
    else:
        stored = 2 * hkv * d * SIZES[case["cache"]]
    read = (hq + 2 * hkv) * d * w + 4 * case["rot"]
    return {"bytes": total * (read + out * d + stored) + 8 * b + 2 * d * w,
            "flops": total * (hq + hkv) * (3 * case["rot"] + 4 * d)}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    s = prepare(case, seed)
    return {"mask": _mask_exact, "keep": _keep_exact, "append": _append_exact}.get(case["op"], _attn_exact)(s)


def _ranges(s):
    """(first row, new tokens, cached tokens before them) of each sequence, as numbers."""
    start, lens = s["indptr"].tolist(), s["lens"].tolist()
    return [(start[i], start[i + 1] - start[i], lens[i] - start[i + 1] + start[i]) for i in range(len(lens))]


def _ancestry(s, window=0, sinks=0):
    """For each token: its position and the drafted tokens that it sees, walked up from it."""
    parents, out = s["parents"].tolist(), []
    for first, n, before in _ranges(s):
        depth = []
        for i in range(n):
            p = parents[first + i]
            depth.append(0 if p < 0 else depth[p] + 1)
            path, j = [], i
            while j >= 0:
                if not window or depth[i] - depth[j] < window or before + depth[j] < sinks:
                    path.append(j)
                j = parents[first + j]
            out.append((before + depth[i], path))
    return out


def _mask_exact(s):
    words = (s["case"]["q_len"] + 31) // 32
    mask, positions = [], []
    for position, path in _ancestry(s, s["case"]["window"], s["case"]["sinks"]):
        positions.append(position)
        row = [sum(1 << (j % 32) for j in path if j // 32 == k) for k in range(words)]
        mask.append([x - (1 << 32) if x >> 31 else x for x in row])
    return {"mask": torch.tensor(mask, dtype=torch.int32, device=DEV), "positions": torch.tensor(positions, dtype=torch.int32, device=DEV)}


def _keep_exact(s):
    page, table, out, lens = s["case"]["page"], s["table"].tolist(), {}, []
    kept, count = s["kept"].tolist(), s["count"].tolist()
    places = []
    for b, (_, n, before) in enumerate(_ranges(s)):
        lens.append(before + count[b])
        for i in range(count[b]):
            a, z = before + kept[b][i], before + i
            places.append((table[b][a // page], a % page, table[b][z // page], z % page))
    for name in ("k", "v"):
        old = s[name]
        out[name] = old.double()
        if places:
            sp, ss, dp, ds = (torch.tensor(x, device=DEV) for x in zip(*places))
            whole = out[name].clone().movedim((1, 3), (0, 1))
            out[name].movedim((1, 3), (0, 1))[dp, ds] = whole[sp, ss]
    out["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    return out


def _attn_exact(s):
    case = s["case"]
    group, d, page, window, sinks = case["hq"] // case["hkv"], case["d"], case["page"], case["window"], case["sinks"]
    trees = _ancestry(s, window, sinks) if case["tree"] else None
    outs, lses = [], []
    for b, (first, n, before) in enumerate(_ranges(s)):
        seen = torch.zeros(n, before + n, dtype=torch.bool, device=DEV)
        for i in range(n):
            position, path = trees[first + i] if case["tree"] else (before + i, list(range(i + 1)))
            lo = max(0, position + 1 - window) if window else 0
            seen[i, min(lo, before):before] = True
            seen[i, :min(sinks, before)] = True
            path = [j for j in path if case["tree"] or before + j >= lo or before + j < sinks]
            seen[i, torch.tensor([before + j for j in path], device=DEV, dtype=torch.long)] = True
        used = seen.any(0).nonzero()[:, 0]
        rows = []
        for pages, scale in ((s["k"], s["scales"][0]), (s["v"], s["scales"][1])):
            raw = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
            x = raw[s["table"][b].long()[used // page], :, used % page]        # [tokens, heads, d]
            x = x.view(torch.float8_e4m3fn) if pages.dtype == torch.float8_e4m3fn else x
            rows.append(x.double().transpose(0, 1).contiguous() * scale)
        q = s["q"][first:first + n].double().view(n, case["hkv"], group, d).permute(1, 0, 2, 3).flatten(1, 2)
        x = torch.bmm(q, rows[0].transpose(1, 2)) / d ** 0.5
        if case["softcap"]:
            x = case["softcap"] * torch.tanh(x / case["softcap"])
        x = x.unflatten(1, (n, group)).masked_fill(~seen[:, used][None, :, None, :], -math.inf)
        lse = torch.logsumexp(x, -1)
        y = torch.bmm(torch.exp(x - lse[..., None]).flatten(1, 2), rows[1])
        outs.append(y.unflatten(1, (n, group)).transpose(0, 1).reshape(n, case["hq"], d))
        lses.append(lse.transpose(0, 1).reshape(n, case["hq"]))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _append_exact(s):
    case = s["case"]
    rot, page = case["rot"], case["page"]
    nv = case["cache"] == "nvfp4"
    slots = torch.cat([torch.arange(before, before + n, device=DEV) for _, n, before in _ranges(s)])
    ids = torch.cat([s["table"][b].long()[torch.arange(before, before + n, device=DEV) // page] for b, (_, n, before) in enumerate(_ranges(s))])
    pos = torch.tensor([p for p, _ in _ancestry(s)], device=DEV) if case["tree"] else slots
    # a rotation is a product of complex numbers
    turn = torch.complex(s["rope"][pos, :rot // 2].double(), s["rope"][pos, rot // 2:].double())[:, None]

    def rotated(x, weight):
        x = x.double()
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["d"] + EPS) * weight.double()
        if case["interleaved"]:
            x[..., :rot] = torch.view_as_real(torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
        else:
            z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
            x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
        return x

    q, k, v = rotated(s["q"], s["q_norm"]), rotated(s["k_new"], s["k_norm"]), s["v_new"].double()
    if not nv:
        out = {}
        for name, x, scale in (("k", k, s["scales"][0]), ("v", v, s["scales"][1])):
            out[name] = s[name].double()
            x = x / scale
            out[name][ids, :, slots % page] = x.clamp(-448, 448) if case["cache"] == "e4m3" else x
        return {"q": q, **out}
    mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    even = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=DEV)  # even codes first: the first of two equally near ones is taken
    values = torch.nn.functional.embedding(s["codes"].int(), s["values"].double())
    sf = s["sf"].double()
    for i, x in enumerate((k, v)):
        blocks = x.unflatten(-1, (-1, 16))
        scale = (blocks.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn).double()
        y = blocks / scale.clamp(min=2.0 ** -30)[..., None]
        near = torch.empty(y.shape, dtype=torch.int64, device=DEV)
        for j in range(0, y.shape[0], 1024):
            near[j:j + 1024] = even[(y[j:j + 1024].abs()[..., None] - mags[even]).abs().argmin(-1)]
        code = torch.where(scale[..., None] > 0, torch.sign(y) * mags[near], 0.0).flatten(-2)
        values[i, ids, :, slots % page] = code.unflatten(-1, (-1, 2))
        sf[i, ids, :, slots % page] = scale
    return {"q": (q / Q_SCALE).clamp(-448, 448), "values": values, "sf": sf}
