"""Plain 64-bit forms of the paged-cache operators, on CPU tensors, written
from their definitions in include/gqa.h: one sequence, one token, one head at
a time where that is the plainest.  Test infrastructure only."""
import math

import torch

E4M3_MAX = 448.0


def positions(total, kv_lens, indptr):
    """(sequence, position) of each token; None for a token that no sequence has."""
    out = [None] * total
    for b, n in enumerate(kv_lens):
        lo, hi = (b, b + 1) if indptr is None else (indptr[b], indptr[b + 1])
        for t in range(lo, min(hi, total)):
            out[t] = (b, n - (hi - t))
    return out


def rotate(x, rope_row, interleaved):
    """One token's heads [H, D] rotated, in x's precision (float64 or float32)."""
    if rope_row is None:
        return x.clone()
    half = rope_row.shape[0] // 2
    c, s = rope_row[:half].to(x.dtype), rope_row[half:].to(x.dtype)
    y = x.clone()
    i = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    j = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = x[:, i], x[:, j]
    y[:, i] = a * c - b * s
    y[:, j] = b * c + a * s
    return y


def rotated(x, rope, where, interleaved, dtype=torch.float64):
    """All tokens' heads rotated to their positions; rows without one are left as they are."""
    y = x.to(dtype).clone()
    for t, w in enumerate(where):
        if w is not None and w[1] >= 0:
            y[t] = rotate(x[t].to(dtype), None if rope is None else rope[w[1]], interleaved)
    return y


def place(pages, rows, where, table, page_size):
    """Scatter rows [T, H, ...] into pages [P, H, page_size, ...] in place."""
    for t, w in enumerate(where):
        if w is not None and w[1] >= 0:
            pages[int(table[w[0], w[1] // page_size]), :, w[1] % page_size] = rows[t]


def gather(pages, table_row, n):
    """The first n tokens of a sequence: [H, n, D] float64."""
    size = pages.shape[2]
    ids = [int(i) for i in table_row[:(n + size - 1) // size]]
    if not ids:
        return torch.zeros(pages.shape[1], 0, pages.shape[3], dtype=torch.float64)
    return torch.cat([pages[i].double() for i in ids], dim=1)[:, :n]


def attention(q, k_pages, v_pages, table, lens, *, q_scale=1.0, k_scale=1.0, v_scale=1.0, window=0, softcap=0.0):
    """out [B, Hq, D], lse [B, Hq] and, for the tolerances, sum_t p_t |v_t| [B, Hq, D] and the
    largest sum_i |q_i k_i| * scale [B, Hq] over the visible tokens; all float64."""
    B, Hq, D = q.shape
    G = Hq // k_pages.shape[1]
    cap_len = table.shape[1] * k_pages.shape[2]
    out, mag = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    lse, reach = torch.full((B, Hq), -math.inf, dtype=torch.float64), torch.zeros(B, Hq, dtype=torch.float64)
    for b in range(B):
        n = max(0, min(int(lens[b]), cap_len))
        first = max(0, n - window) if window else 0
        if n == 0:
            continue
        k, v = gather(k_pages, table[b], n)[:, first:], gather(v_pages, table[b], n)[:, first:]
        for h in range(Hq):
            x = q[b, h].double()
            f = q_scale * k_scale / math.sqrt(D)
            s = (k[h // G] @ x) * f
            reach[b, h] = (k[h // G].abs() @ x.abs()).max() * abs(f)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            lse[b, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[b, h])
            out[b, h] = (p @ v[h // G]) * v_scale
            mag[b, h] = (p @ v[h // G].abs()) * v_scale
    return out, lse, mag, reach


def visible_magnitude(v_pages, table, lens, q_heads, *, v_scale=1.0, window=0, **_):
    """sum_t |v_t| * v_scale over the visible tokens, [B, Hq, D]."""
    cap_len = table.shape[1] * v_pages.shape[2]
    rows = []
    for b in range(len(lens)):
        n = max(0, min(int(lens[b]), cap_len))
        v = gather(v_pages, table[b], n)[:, max(0, n - window) if window else 0:]
        rows.append(v.abs().sum(1).repeat_interleave(q_heads // v_pages.shape[1], 0) * v_scale)
    return torch.stack(rows)


def check_attention(got, got_lse, q, k_pages, v_pages, table, lens, **kw):
    """The bound, in its parts.  A score is a sum of D products over at most 16 chained f32 additions
    of a tensor-core step each (D <= 256): |error| <= 16 * 2^-23 * sum |q_i k_i| * scale; capping adds
    at most 4 roundings of an exponential's 2^-22 times the cap; the logarithm and the scale 2^-20 (1 +
    |lse|).  A weight is off by twice the scores' error (its own and the sum's) and by its rounding for
    the product with V: 2^-16 for a pair of terms, 2^-11 for the one f16 term of E4M3 pages and bf16
    queries.  An f16 weight (f16 and E4M3 pages) also has a floor: the largest weight of a warp's keys is 2^14
    and f16's spacing is nowhere below 2^-24, so that a weight is off by half of it, 2^-25, at most: 2^-39
    of the largest weight and so of the weights' sum, whatever its own size.  (It shows where an output's large
    weights all meet v = 0.)  An output is a weighted sum, off by the weights' errors times |v|, and is
    rounded once by half a step of its type."""
    out, lse, mag, reach = attention(q.cpu(), k_pages.cpu(), v_pages.cpu(), table.cpu(), lens.cpu(), **kw)
    s_err = 2.0 ** -19 * reach + 2.0 ** -20 * kw.get("softcap", 0.0) + 2.0 ** -20
    w = 2.0 ** -11 if k_pages.dtype == torch.float8_e4m3fn and q.dtype == torch.bfloat16 else 2.0 ** -16
    fin = torch.finfo(got.dtype)
    tol = fin.eps / 2 * out.abs() + (1 + fin.eps) * (w + 2 * s_err)[..., None] * mag + fin.smallest_normal * fin.eps
    if v_pages.dtype != torch.bfloat16:
        tol += 2.0 ** -39 * visible_magnitude(v_pages.cpu(), table.cpu(), lens.cpu(), q.shape[1], **kw)
    err = (got.cpu().double() - out).abs()
    assert torch.isfinite(got.cpu().double()).all()
    assert (err <= tol).all(), f"out: worst {float((err / tol).max()):.2f} of the bound, |err| {float(err.max()):.3g}"
    if got_lse is not None:
        g = got_lse.cpu().double()
        empty = torch.isinf(lse)
        assert torch.equal(torch.isinf(g), empty) and (g[empty] < 0).all()
        e = (g - lse).abs()[~empty]
        t = (s_err + 2.0 ** -20 * lse.abs().clamp(max=1e30))[~empty]
        assert (e <= t).all(), f"lse: worst {float((e / t).max()):.2f} of the bound"


def e4m3_values(x):
    """float64 nearest E4M3 values (ties to even), saturating."""
    return x.clamp(-E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn).double()


E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_decode(packed):
    """[..., n] bytes -> [..., 2 n] values."""
    code = torch.stack([packed & 15, packed >> 4], dim=-1).flatten(-2).long()
    return torch.where(code >= 8, -E2M1[code & 7], E2M1[code & 7])


def nvfp4_quantise(x):
    """x [..., D] float32 -> (values [..., D], scales [..., D / 16]) by the definition, in float32."""
    blocks = x.unflatten(-1, (-1, 16))
    amax = blocks.abs().amax(-1)
    sf = (amax / torch.tensor(6.0)).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn).float()
    ok = sf > 0
    y = torch.where(ok[..., None], blocks / torch.where(ok, sf, 1.0)[..., None], 0.0)
    a = y.abs().clamp(max=6.0)
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7])  # even codes first: of two equally near, the even one
    near = order[(a.double()[..., None] - E2M1[order].double()).abs().argmin(-1)]
    return (torch.copysign(E2M1[near], y)).flatten(-2), sf
