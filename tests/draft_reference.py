"""Plain 64-bit forms of the operators of drafted tokens, on CPU tensors, written
from their definitions in include/gqa.h, one token at a time.  Test infrastructure only."""
import math

import torch

import paged_reference as R


def normed(x, weight, eps):
    """[T, H, D] float64: each head by its root mean square, weighted."""
    x = x.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()


def trees(parents, indptr, lens, window=0, sinks=0):
    """For each drafted token: (position, the numbers of the tokens of its draft that it sees)."""
    out = []
    for b in range(len(lens)):
        lo, n = indptr[b], indptr[b + 1] - indptr[b]
        base, depth = lens[b] - n, []
        for i in range(n):
            p = parents[lo + i]
            depth.append(depth[p] + 1 if p >= 0 else 0)
            seen, j = set(), i
            while j >= 0:
                if not window or depth[i] - depth[j] < window or base + depth[j] < sinks:
                    seen.add(j)
                j = parents[lo + j]
            out.append((base + depth[i], seen))
    return out


def words_of(seen, words):
    """The bits of a set as int32 words."""
    row = [sum(1 << (j % 32) for j in seen if j // 32 == w) for w in range(words)]
    return [x - (1 << 32) if x >= 1 << 31 else x for x in row]


def visible_one(n, window, sinks):
    """The cache places that one new token of a sequence of n tokens sees."""
    first = max(0, n - window) if window else 0
    return sorted(set(range(first, n)) | set(range(min(sinks, n))))


def visible_rows(indptr, lens, window=0, sinks=0, mask=None, positions=None):
    """For each row: the cache places that it sees.  Without a mask the drafted tokens are a chain."""
    out = []
    for b in range(len(lens)):
        lo, n = indptr[b], indptr[b + 1] - indptr[b]
        base = lens[b] - n
        for i in range(n):
            if mask is None:
                at = base + i
                out.append([t for t in range(0, at + 1) if not window or t > at - window or t < sinks])
                continue
            p = max(base, positions[lo + i]) if window else 0
            seen = [t for t in range(0, max(0, base)) if not window or t > p - window or t < sinks]
            bits = [j for j in range(min(n, 32 * len(mask[lo + i]))) if mask[lo + i][j // 32] >> (j % 32) & 1]
            out.append(seen + [base + j for j in bits if base + j >= 0])
    return out


def attention(q, k_pages, v_pages, tables, visible, *, q_scale=1.0, k_scale=1.0, v_scale=1.0, softcap=0.0):
    """Row t of q [T, Hq, D] over the tokens visible[t] of the sequence whose block table row is tables[t]: out
    [T, Hq, D], lse [T, Hq] and, for the tolerances, sum p |v|, the largest sum |q k| * scale and sum |v|; float64."""
    T, Hq, D = q.shape
    G, size = Hq // k_pages.shape[1], k_pages.shape[2]
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64)
    out, mag, all_v, reach = zero(T, Hq, D), zero(T, Hq, D), zero(T, Hq, D), zero(T, Hq)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    f = q_scale * k_scale / math.sqrt(D)
    k_pages, v_pages = k_pages.double(), v_pages.double()
    for t in range(T):
        if not visible[t]:
            continue
        at = torch.tensor(visible[t])
        ids, slot = tables[t].long()[at // size], at % size
        k, v = (p[ids, :, slot].transpose(0, 1) for p in (k_pages, v_pages))  # [Hkv, n, D]
        k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
        x = q[t].double()
        s = torch.einsum("hd,hnd->hn", x, k) * f
        reach[t] = torch.einsum("hd,hnd->hn", x.abs(), k.abs()).amax(-1) * abs(f)
        if softcap:
            s = softcap * torch.tanh(s / softcap)
        lse[t] = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[t][:, None])
        out[t] = torch.einsum("hn,hnd->hd", p, v) * v_scale
        mag[t] = torch.einsum("hn,hnd->hd", p, v.abs()) * v_scale
        all_v[t] = v.abs().sum(1) * v_scale
    return out, lse, mag, reach, all_v


def check_attention(got, got_lse, q, k_pages, v_pages, tables, visible, **kw):
    """The bound of paged_reference.check_attention (its docstring derives it) for rows that see any set of tokens,
    and, for more than 1000 of them, the f32 additions of the product with V: one for 16 tokens, each off by 2^-23
    of the sum at most (half of that if it rounds to nearest)."""
    out, lse, mag, reach, all_v = attention(q.cpu(), k_pages.cpu(), v_pages.cpu(), tables, visible, **kw)
    s_err = 2.0 ** -19 * reach + 2.0 ** -20 * kw.get("softcap", 0.0) + 2.0 ** -20
    w = 2.0 ** -16 + 2.0 ** -23 * max([len(x) for x in visible] + [0]) / 16
    fin = torch.finfo(got.dtype)
    tol = fin.eps / 2 * out.abs() + (1 + fin.eps) * (w + 2 * s_err)[..., None] * mag + fin.smallest_normal * fin.eps
    if v_pages.dtype != torch.bfloat16:
        tol += 2.0 ** -39 * all_v
    g = got.cpu().double()
    assert torch.isfinite(g).all()
    err = (g - out).abs()
    assert (err <= tol).all(), f"out: worst {float((err / tol).max()):.2f} of the bound, |err| {float(err.max()):.3g}"
    if got_lse is not None:
        l = got_lse.cpu().double()
        empty = torch.isinf(lse)
        assert torch.equal(torch.isinf(l), empty) and (l[empty] < 0).all()
        e = (l - lse).abs()[~empty]
        t = (s_err + 2.0 ** -20 * lse.abs().clamp(max=1e30))[~empty]
        assert (e <= t).all(), f"lse: worst {float((e / t).max()):.2f} of the bound"
