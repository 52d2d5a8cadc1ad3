"""The cache operators as measured cases: appending rotated keys and values to a paged cache, and
attention of one new token per sequence over such a cache.

    gqa_paged_append    rotary embedding of q and k, and the write of k and v into 16-bit or E4M3 pages
    nvfp4_paged_append  the same into NVFP4 pages (E2M1 codes, E4M3 block scales), q leaving as E4M3
    gqa_paged_attn      one query token per sequence over 16-bit or E4M3 pages, split over the length

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
K_SCALE, V_SCALE = 0.0625, 0.03125  # E4M3 pages: stored value = value / scale
Q_SCALE = 0.03125                   # NVFP4 path: E4M3 query = query / scale


# ------------------------------------------------------------------ cases ---

def _append(name, type, cache, batch, q_len, kv_len, hq, hkv, d, rot, page, layout, interleaved, ragged):
    c = dict(op="append", type=type, cache=cache, batch=batch, q_len=q_len, kv_len=kv_len, hq=hq, hkv=hkv, d=d, rot=rot,
             page=page, layout=layout, interleaved=interleaved, ragged=ragged)
    return dict(name=name, **c) if name else c


def _attn(name, type, cache, batch, kv_len, hq, hkv, d, page, layout, window, softcap, ragged):
    c = dict(op="attn", type=type, cache=cache, batch=batch, kv_len=kv_len, hq=hq, hkv=hkv, d=d, page=page, layout=layout,
             window=window, softcap=softcap, ragged=ragged)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one sequence, one new token: a chat turn's decode step, where the launch is what counts
        _append("append_b1", "f16", "f16", 1, 1, 1024, 32, 8, 128, 128, 64, "hnd", False, False),
        # a decode step of a full serving batch into an E4M3 cache of small token-major pages
        _append("append_b256_e4m3", "bf16", "e4m3", 256, 1, 509, 32, 8, 128, 128, 16, "nhd", False, True),
        # prompts: batch 4 of 2048 tokens
        _append("append_b4_q2048", "bf16", "bf16", 4, 2048, 2048, 32, 8, 128, 128, 64, "hnd", False, False),
        # chunks of long prompts, ragged, partial interleaved rotation, head dim 256
        _append("append_b7_q4099", "f16", "f16", 7, 4099, 9001, 16, 4, 256, 64, 32, "hnd", True, True),
        # NVFP4: a short ragged chunk, and the prompts of the context workload
        _append("nvfp4_b3_q201", "bf16", "nvfp4", 3, 201, 333, 32, 8, 128, 128, 64, "hnd", False, True),
        _append("nvfp4_b4_q2048", "bf16", "nvfp4", 4, 2048, 2048, 32, 8, 128, 128, 64, "hnd", False, False),
        # the smallest decode configuration: lengths 1 and 200
        _attn("attn_b2_cap200", "f16", "f16", 2, 200, 32, 8, 128, 64, "hnd", 0, 0.0, True),
        # one sequence with a long context: few rows, so the length has to be split
        _attn("attn_b1_kv32768", "bf16", "bf16", 1, 32768, 32, 8, 128, 16, "hnd", 0, 0.0, False),
        # a serving batch of ragged lengths up to 8192
        _attn("attn_b64_kv8192", "bf16", "bf16", 64, 8192, 32, 8, 128, 64, "hnd", 0, 0.0, True),
        # the same kind of batch with eight query heads per KV head over an E4M3 cache
        _attn("attn_b48_e4m3", "bf16", "e4m3", 48, 16001, 64, 8, 128, 16, "nhd", 0, 0.0, True),
        # sliding window, capped scores, head dim 256, two query heads per KV head
        _attn("attn_b33_window", "bf16", "bf16", 33, 6007, 16, 8, 256, 32, "nhd", 4096, 50.0, True),
        # long contexts: 8 sequences of 131072 tokens
        _attn("attn_b8_kv131072", "f16", "f16", 8, 131072, 32, 8, 128, 64, "hnd", 0, 0.0, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = [(32, 8), (64, 8), (16, 8), (8, 8), (28, 4), (16, 1), (5, 1), (40, 2), (12, 12)]
    page, layout = rng.choice([16, 32, 64, 128]), rng.choice(["hnd", "nhd"])
    kind = rng.choice(["append", "append", "nvfp4", "attn", "attn", "attn"])
    if kind == "nvfp4":
        batch = _log(rng, 1, 24)
        q_len = _log(rng, 1, 8192 // batch)
        kv_len = q_len + rng.choice([0, rng.randint(0, 200)])
        return _append(None, rng.choice(["f16", "bf16"]), "nvfp4", batch, q_len, kv_len, 32, 8, 128, rng.choice([128, 128, 64]), 64,
                       "hnd", rng.random() < 0.3, batch > 1 and rng.random() < 0.6)
    type = rng.choice(["f16", "bf16"])
    cache = rng.choice([type, type, "e4m3"])
    hq, hkv = rng.choice(heads)
    d = rng.choice([64, 128, 128, 256])
    if kind == "append":
        room = min(16384, 200_000_000 // ((hq + 2 * hkv) * d * 2))
        batch = _log(rng, 1, min(256, room))
        q_len = rng.choice([1, _log(rng, 1, max(1, room // batch))])
        kv_len = q_len + _log(rng, 1, 400) - 1
        return _append(None, type, cache, batch, q_len, kv_len, hq, hkv, d, rng.choice([r for r in (32, 64, 128, 256) if r <= d]),
                       page, layout, rng.random() < 0.4, batch > 1 and rng.random() < 0.6)
    room = 4_000_000_000 // (2 * hkv * d * 2)
    batch = _log(rng, 1, 256)
    kv_len = _log(rng, 1, max(2, min(131072, room // batch)))
    return _attn(None, type, cache, batch, kv_len, hq, hkv, d, page, layout, rng.choice([0, 0, 0, _log(rng, 16, 4096)]),
                 rng.choice([0.0, 0.0, 30.0]), batch > 1 and rng.random() < 0.7)


def _lengths(case, key):
    """Lengths of the sequences: all alike, or evenly spread from 1 to the case's."""
    b, n = case["batch"], case[key]
    if not case["ragged"] or b == 1:
        return [n] * b
    return [1 + (n - 1) * i // (b - 1) for i in range(b)]


# ----------------------------------------------------------------- inputs ---

def _pages(gen, dtype, num, hkv, page, d, layout):
    """[num, hkv, page, d] (a view where the storage is token-major), filled as an older cache is."""
    shape = (num, page, hkv, d) if layout == "nhd" else (num, hkv, page, d)
    t = torch.empty(shape, dtype=dtype, device=DEV)
    for i in range(0, num, 4096):
        x = torch.empty((min(4096, num - i),) + shape[1:], dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
        t[i:i + 4096] = (x * 16).clamp(-448, 448).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)
    return t.permute(0, 2, 1, 3) if layout == "nhd" else t


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


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    b, hq, hkv, d, page = case["batch"], case["hq"], case["hkv"], case["d"], case["page"]
    order = torch.randperm(b, generator=gen, device=DEV).tolist()
    dtype = DTYPES[case["type"]]
    s = dict(case=case)
    if case["op"] == "attn":
        lens = [_lengths(case, "kv_len")[i] for i in order]
        s["table"], num = _table(gen, lens, page)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q"] = (torch.empty(b, hq, d, device=DEV).normal_(generator=gen) * 1.5).to(dtype)
        s["k"] = _pages(gen, DTYPES[case["cache"]], num, hkv, page, d, case["layout"])
        s["v"] = _pages(gen, DTYPES[case["cache"]], num, hkv, page, d, case["layout"])
        s["scales"] = (K_SCALE, V_SCALE) if case["cache"] == "e4m3" else (1.0, 1.0)
        return s
    new = [_lengths(case, "q_len")[i] for i in order]
    lens = [n + case["kv_len"] - case["q_len"] for n in new]  # the same number of cached tokens before each chunk
    s["table"], num = _table(gen, lens, page)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["indptr"] = torch.tensor([0] + new, dtype=torch.int32, device=DEV).cumsum(0).to(torch.int32)
    # q, k and v as a fused projection leaves them: slices of one row per token
    qkv = torch.empty(sum(new), hq + 2 * hkv, d, dtype=dtype, device=DEV).normal_(generator=gen)
    qkv[:, hq:hq + hkv, ::16] *= 4  # keys have channels that stand out
    s["q"], s["k_new"], s["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    s["rope"] = _rope_table(max(lens), case["rot"])
    if case["cache"] == "nvfp4":
        # codes [K|V, pages, heads, tokens, d / 2] and scales [K|V, pages, heads, tokens, d / 16]
        s["codes"] = torch.randint(0, 256, (2, num, hkv, page, d // 2), generator=gen, device=DEV, dtype=torch.uint8)
        s["sf"] = torch.rand(2, num, hkv, page, d // 16, generator=gen, device=DEV).add(0.1).to(torch.float8_e4m3fn)
        mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
        vals = torch.cat([mags, -mags]).half()
        byte = torch.arange(256, device=DEV)
        s["values"] = torch.stack([vals[byte % 16], vals[byte // 16]], dim=1)  # the two values of a byte
    else:
        s["k"] = _pages(gen, DTYPES[case["cache"]], num, hkv, page, d, case["layout"])
        s["v"] = _pages(gen, DTYPES[case["cache"]], num, hkv, page, d, case["layout"])
        s["scales"] = (K_SCALE, V_SCALE) if case["cache"] == "e4m3" else (1.0, 1.0)
    return s


# ------------------------------------------------------------------- run ----

def run(state):
    case = state["case"]
    if case["op"] == "attn":
        return _attn_own(state) if own else _attn_plain(state)
    if case["cache"] == "nvfp4":
        q = _nvfp4_own(state) if own else _nvfp4_plain(state)
        # the codes as the values that they stand for
        values = torch.nn.functional.embedding(state["codes"].int(), state["values"])
        return {"q": q, "values": values, "sf": state["sf"]}
    q = _append_own(state) if own else _append_plain(state)
    return {"q": q, "k": state["k"], "v": state["v"]}


def _append_own(s):
    import gqa_attention_kv_split_gb300 as gqa
    case = s["case"]
    return gqa.gqa_paged_append(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"],
                                qo_indptr=None if case["q_len"] == 1 else s["indptr"], rope=s["rope"],
                                interleaved=case["interleaved"], k_scale=s["scales"][0], v_scale=s["scales"][1])


def _nvfp4_own(s):
    import gqa_attention_kv_split_gb300 as gqa
    q = gqa.nvfp4_paged_append(s["q"], s["k_new"], s["v_new"], s["codes"][0], s["sf"][0], s["codes"][1], s["sf"][1], s["table"],
                               s["indptr"], s["lens"], rope=s["rope"], interleaved=s["case"]["interleaved"], q_scale=Q_SCALE)
    return q.view(torch.float8_e4m3fn)


def _attn_own(s):
    import gqa_attention_kv_split_gb300 as gqa
    case = s["case"]
    lse = torch.empty(case["batch"], case["hq"], dtype=torch.float32, device=s["q"].device)
    out = gqa.gqa_paged_attn(s["q"], s["k"], s["v"], s["table"], s["lens"], lse=lse, window=case["window"], softcap=case["softcap"],
                             k_scale=s["scales"][0], v_scale=s["scales"][1])
    return {"out": out, "lse": lse}


def _places(s):
    """Position, page and slot of each new token."""
    t = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(s["indptr"][1:].contiguous(), t.int(), right=True)
    pos = t - s["indptr"][seq + 1] + s["lens"][seq]
    page = s["case"]["page"]
    return pos, s["table"][seq, pos // page].long(), pos % page


def _rotate(x, cos, sin, interleaved):
    """Rotary embedding of the first 2 * cos.shape[-1] elements of each head, in x's type."""
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
    """q and k rotated to their positions, and v, in 32 bits."""
    half = s["case"]["rot"] // 2
    cs = s["rope"][pos]
    cos, sin, inter = cs[:, :half], cs[:, half:], s["case"]["interleaved"]
    return _rotate(s["q"].float(), cos, sin, inter), _rotate(s["k_new"].float(), cos, sin, inter), s["v_new"].float()


def _rounded(x, dtype, scale):
    """x / scale in `dtype`; E4M3 saturates."""
    if scale != 1.0:
        x = x * torch.tensor(1.0 / scale, dtype=torch.float32, device=x.device)
    return x.clamp(-448, 448).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)


def _append_plain(s):
    pos, page, slot = _places(s)
    q, k, v = _turned(s, pos)
    for pages, x, scale in ((s["k"], k, s["scales"][0]), (s["v"], v, s["scales"][1])):
        y = _rounded(x, pages.dtype, scale)
        if pages.dtype == torch.float8_e4m3fn:
            pages, y = pages.view(torch.uint8), y.view(torch.uint8)
        pages[page, :, slot] = y
    return q.to(s["q"].dtype)


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


def _attn_plain(s):
    case = s["case"]
    b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    k = _gathered(s["k"], s["table"])
    q = s["q"].float().view(b, hkv, hq // hkv, d)
    x = torch.matmul(q, k.transpose(-1, -2)) * (s["scales"][0] / math.sqrt(d))  # [b, hkv, group, tokens]
    del k
    if case["softcap"]:
        x = torch.tanh(x / case["softcap"]) * case["softcap"]
    t, lens = torch.arange(x.shape[-1], device=DEV)[None, :], s["lens"][:, None]
    seen = t < lens
    if case["window"]:
        seen = seen & (t >= lens - case["window"])
    seen = seen[:, None, None, :]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.where(seen, torch.exp(x - m), 0.0)
    total = e.sum(-1, keepdim=True)
    v = _gathered(s["v"], s["table"])
    v = torch.where(seen[:, :, 0, :, None], v, 0.0)
    out = torch.matmul(e, v) / total * s["scales"][1]
    out = torch.where(total > 0, out, 0.0)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)
    return {"out": out.view(b, hq, d).to(s["q"].dtype), "lse": lse.view(b, hq)}


# ------------------------------------------------------------------- work ---

def work(case):
    b, hq, hkv, d, page = case["batch"], case["hq"], case["hkv"], case["d"], case["page"]
    w = SIZES[case["type"]]
    if case["op"] == "attn":
        lens = [min(n, case["window"]) if case["window"] else n for n in _lengths(case, "kv_len")]
        n = sum(lens)
        table = sum((x + page - 1) // page for x in lens) * 4
        return {"bytes": 2 * n * hkv * d * SIZES[case["cache"]] + 2 * b * hq * d * w + 4 * b * hq + 4 * b + table,
                "flops": 4 * n * hq * d}
    n = sum(_lengths(case, "q_len"))
    out = w * hq
    if case["cache"] == "nvfp4":
        stored = 2 * hkv * d * (0.5 + 1 / 16)
        out = hq
    else:
        stored = 2 * hkv * d * SIZES[case["cache"]]
    read = (hq + 2 * hkv) * d * w + 4 * case["rot"]
    return {"bytes": n * (read + out * d + stored) + 4 * b * 2, "flops": 3 * n * (hq + hkv) * case["rot"]}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _attn_exact(s)
    return _append_exact(s)


def _attn_exact(s):
    case = s["case"]
    group, d = case["hq"] // case["hkv"], case["d"]
    outs, lses = [], []
    for i, n in enumerate(s["lens"].tolist()):
        first = max(0, n - case["window"]) if case["window"] else 0
        ids = s["table"][i, :(n + case["page"] - 1) // case["page"]].long()
        rows = []
        for pages, scale in ((s["k"], s["scales"][0]), (s["v"], s["scales"][1])):
            e4m3 = pages.dtype == torch.float8_e4m3fn
            x = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() if e4m3 else pages[ids].double()
            rows.append(x.transpose(0, 1).reshape(case["hkv"], -1, d)[:, first:n] * scale)
        q = s["q"][i].double().view(case["hkv"], group, d)
        x = torch.einsum("hgd,htd->hgt", q, rows[0]) / d ** 0.5
        if case["softcap"]:
            x = case["softcap"] * torch.tanh(x / case["softcap"])
        lse = torch.logsumexp(x, -1)
        outs.append(torch.einsum("hgt,htd->hgd", torch.exp(x - lse[..., None]), rows[1]).reshape(case["hq"], d))
        lses.append(lse.reshape(-1))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _append_exact(s):
    case = s["case"]
    rot, page = case["rot"], case["page"]
    nv = case["cache"] == "nvfp4"
    start, lens, table = s["indptr"].tolist(), s["lens"].tolist(), s["table"]
    pos = torch.cat([torch.arange(lens[i] - (start[i + 1] - start[i]), lens[i], device=DEV) for i in range(case["batch"])])
    ids = torch.cat([table[i].long()[torch.arange(lens[i] - (start[i + 1] - start[i]), lens[i], device=DEV) // page] for i in range(case["batch"])])
    # a rotation is a product of complex numbers
    turn = torch.complex(s["rope"][pos, :rot // 2].double(), s["rope"][pos, rot // 2:].double())[:, None]

    def rotated(x):
        x = x.double().clone()
        if case["interleaved"]:
            x[..., :rot] = torch.view_as_real(torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
        else:
            z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
            x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
        return x

    q, k, v = rotated(s["q"]), rotated(s["k_new"]), s["v_new"].double()
    if not nv:
        out = {}
        for name, x, scale in (("k", k, s["scales"][0]), ("v", v, s["scales"][1])):
            out[name] = s[name].double()
            x = x / scale
            out[name][ids, :, pos % page] = x.clamp(-448, 448) if case["cache"] == "e4m3" else x
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
        values[i, ids, :, pos % page] = code.unflatten(-1, (-1, 2))
        sf[i, ids, :, pos % page] = scale
    return {"q": (q / Q_SCALE).clamp(-448, 448), "values": values, "sf": sf}
