"""GPU: the appends with norms of the heads and given positions, against their plain 64-bit forms."""
import pytest
import torch

import draft_reference as DR
import gqa_attention_kv_split_gb300 as gqa
import paged_reference as R
from test_gpu_paged_append import Case, rope_table

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


def weights(d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [(torch.rand(d, generator=g) * 2 + 0.25).to(dtype) for _ in range(2)]


def turned(x, rope, rows, interleaved):
    """[T, H, D] float64 rotated with the given rows of the table (None: not rotated)."""
    y = x.clone()
    for t, r in enumerate(rows):
        if r is not None:
            y[t] = R.rotate(x[t], None if rope is None else rope[r], interleaved)
    return y


def magnitude(x, rope, rows, interleaved):
    """|x c| + |y s| of each rotated pair, |x| of the others."""
    if rope is None:
        return x.abs()
    half = rope.shape[1] // 2
    sign = torch.cat([torch.ones(half), -torch.ones(half)])
    return turned(x.abs(), rope.abs() * sign, rows, interleaved).abs() + x.abs()


def bound(x, mag, dtype, inv=1.0):
    """Half a step of the stored type, and 2^-19 of the terms: the sum of at most 256 squares in 16 additions a
    thread and 4 levels of a tree, halved by the root (10 * 2^-24), the reciprocal root's 2 steps (2^-22), two products
    for the weight and two roundings and a sum for the rotation (5 * 2^-24): 19 * 2^-24 < 2^-19."""
    slack = 2.0 ** -19 * mag * inv
    if dtype == E4M3:
        return torch.maximum(2.0 ** -4 * x.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64)) * (1 + 2.0 ** -10) + slack
    f = torch.finfo(dtype)
    return f.eps / 2 * x.abs() * (1 + f.eps) + slack + f.smallest_normal * f.eps


def check(c, interleaved=False, scales=(1.0, 1.0), which="qk", wtype=None, positions=None, eps=1e-6, one_each=False, in_place=False):
    a = c.device()
    d = c.q.shape[2]
    wq, wk = weights(d, wtype or c.q.dtype, d)
    kp, vp = c.k_pages.to(DEV), c.v_pages.to(DEV)
    if one_each:
        a["qo_indptr"] = None
    q_out = a["q"] if in_place else torch.full((c.total,) + c.q.shape[1:], 7.0, dtype=c.q.dtype, device=DEV)
    got = gqa.gqa_paged_append(**a, k_pages=c.view(kp), v_pages=c.view(vp), interleaved=interleaved, k_scale=scales[0],
                               v_scale=scales[1], q_out=q_out, q_norm=wq.to(DEV) if "q" in which else None,
                               k_norm=wk.to(DEV) if "k" in which else None, norm_eps=eps,
                               positions=None if positions is None else torch.tensor(positions, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    live = [w is not None and w[1] >= 0 for w in c.where]
    rows = [(w[1] if positions is None else positions[t]) if live[t] else None for t, w in enumerate(c.where)]
    live = torch.tensor(live)
    q = DR.normed(c.q, wq, eps) if "q" in which else c.q.double()
    k = DR.normed(c.k, wk, eps) if "k" in which else c.k.double()
    want = turned(q, c.rope, rows, interleaved)
    err = (got.cpu().double() - want)[live].abs()
    tol = bound(want, magnitude(q, c.rope, rows, interleaved), c.q.dtype)[live]
    assert (err <= tol).all(), f"q: {float((err / tol).max())} of the bound"
    if not in_place:
        assert (got.cpu()[~live] == 7.0).all()
    for name, x, mag, pages, scale, dev in (
            ("k", turned(k, c.rope, rows, interleaved), magnitude(k, c.rope, rows, interleaved), c.k_pages, scales[0], kp),
            ("v", c.v.double(), c.v.double().abs(), c.v_pages, scales[1], vp)):
        x = x / scale
        if c.cache == E4M3:
            x = x.clamp(-448, 448)
        want, tol = pages.double().clone(), torch.zeros(pages.shape, dtype=torch.float64)
        R.place(c.view(want), x, c.where, c.table, c.page)
        R.place(c.view(tol), bound(x, mag, c.cache, 1 / scale), c.where, c.table, c.page)
        e = (dev.cpu().double() - want).abs()
        assert (e <= tol).all(), f"{name}: {float(e.max())}"  # untouched slots: exactly as they were


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (64, 16, False), (64, 48, True), (128, 128, False), (128, 64, True),
                                         (128, 0, False), (256, 256, False), (256, 80, False), (256, 256, True)])
def test_matches_plain_form(dtype, d, rot, inter):
    check(Case([5, 1, 40], [5, 17, 40], d=d, rot=rot, dtype=dtype, seed=d + rot), interleaved=inter)


@pytest.mark.parametrize("which", ["q", "k", "qk"])
@pytest.mark.parametrize("wtype", [BF16, torch.float32])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_one_norm_or_both(which, wtype, layout):
    check(Case([3, 0, 9], [20, 0, 9], hq=5, hkv=5, d=128, rot=64, layout=layout, seed=3), which=which, wtype=wtype)


@pytest.mark.parametrize("hq,hkv,page", [(1, 1, 16), (28, 4, 64), (7, 7, 5), (40, 2, 128), (3, 1, 1)])
def test_heads_and_pages(hq, hkv, page):
    check(Case([1] * 12, list(range(1, 13)), hq=hq, hkv=hkv, d=128, page=page, seed=hq), one_each=True)
    check(Case([33, 2], [40, 2], hq=hq, hkv=hkv, d=64, page=page, seed=hq, pad=3))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_e4m3_pages(dtype, d):
    check(Case([5, 20], [9, 33], d=d, dtype=dtype, cache=E4M3, seed=d, spread=3.0), scales=(0.02, 0.05))


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_positions_choose_the_angles(cache):
    """A tree's tokens: places in the cache one after the other, positions by depth."""
    c = Case([6, 1, 3], [46, 1, 90], d=128, rot=128, cache=cache, seed=9)
    check(c, positions=[40, 40, 41, 41, 42, 41, 0, 87, 88, 88], scales=(0.02, 0.05) if cache == E4M3 else (1.0, 1.0))
    check(c, positions=[5, 0, 89, 3, 3, 3, 7, 1, 2, 80], which="", scales=(0.02, 0.05) if cache == E4M3 else (1.0, 1.0))


def test_in_place_and_large_batches():
    check(Case([1] * 700, [1 + i % 50 for i in range(700)], hq=8, hkv=2, d=128, seed=4), one_each=True, in_place=True)
    check(Case([900, 300], [900, 400], hq=4, hkv=2, d=128, seed=5))


def test_small_and_large_heads():
    """Heads far below eps's root, of zeros alone, and of squares up to 2^100."""
    for spread, eps in ((1e-6, 1e-6), (0.0, 1e-6), (2.0 ** 50, 1e-6), (1e-3, 0.0)):
        check(Case([4], [4], d=64, rot=64, dtype=BF16, seed=6, spread=spread), eps=eps)


def test_a_nan_stays_in_its_head():
    c = Case([2], [2], hq=3, hkv=2, d=64, seed=7)
    a = c.device()
    a["q"][1, 2, 5] = float("nan")
    kp, vp = c.k_pages.to(DEV), c.v_pages.to(DEV)
    w = torch.ones(64, dtype=BF16, device=DEV)
    got = gqa.gqa_paged_append(**a, k_pages=kp, v_pages=vp, q_norm=w, k_norm=w)
    bad = got.isnan()
    assert bad[1, 2].all() and int(bad.sum()) == 64 and not kp.isnan().any()


def test_positions_outside_the_table_are_flagged():
    c = Case([4], [4], d=64, seed=8)
    a = c.device()
    kp, vp = c.k_pages.to(DEV), c.v_pages.to(DEV)
    before = kp.clone()
    q_out = torch.full_like(c.q, 7.0, device=DEV).contiguous()
    gqa.gqa_paged_append(**a, k_pages=kp, v_pages=vp, q_out=q_out,
                         positions=torch.tensor([0, -1, 4, 2 ** 31 - 1], dtype=torch.int32, device=DEV))
    assert gqa.gqa_check_device_errors(0) == 2
    assert (q_out[1:] == 7.0).all() and not (q_out[0] == 7.0).any()
    assert int((kp != before).any(-1).sum()) == 2  # the two heads of the one token


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.mark.parametrize("rot,inter,tree", [(128, False, False), (64, False, True), (128, True, True), (0, False, False)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_nvfp4(dtype, rot, inter, tree):
    """Scales and codes are the nearest ones to values off by 2^-19 of their terms."""
    c = Case([7, 1, 70], [7, 30, 100], hq=32, hkv=8, d=128, page=64, rot=rot, dtype=dtype, seed=rot)
    a = c.device()
    wq, wk = weights(128, torch.float32, 11)
    z = [torch.full((c.num, 8, 64, w), 0x55, dtype=torch.uint8, device=DEV) for w in (64, 8, 64, 8)]
    rows = [w[1] for w in c.where]
    positions = None
    if tree:
        rows = [max(0, r - t % 3) for t, r in enumerate(rows)]
        positions = torch.tensor(rows, dtype=torch.int32, device=DEV)
    q = gqa.nvfp4_paged_append(a["q"], a["k"], a["v"], *z, a["block_table"], a["qo_indptr"], a["kv_lens"], rope=a["rope"],
                               interleaved=inter, q_scale=0.05, q_norm=wq.to(DEV), k_norm=wk.to(DEV), positions=positions)
    torch.cuda.synchronize()
    xq, xk = DR.normed(c.q, wq, 1e-6), DR.normed(c.k, wk, 1e-6)
    want = (turned(xq, c.rope, rows, inter) / 0.05).clamp(-448, 448)
    got = q.view(E4M3).cpu().double()
    assert ((got - want).abs() <= bound(want, magnitude(xq, c.rope, rows, inter), E4M3, 20.0)).all()
    grid = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64)
    levels = torch.arange(0, 127, dtype=torch.uint8).view(E4M3).double()  # the finite positive E4M3 numbers
    for x, mag, codes, sf in ((turned(xk, c.rope, rows, inter), magnitude(xk, c.rope, rows, inter), z[0], z[1]),
                              (c.v.double(), c.v.double().abs(), z[2], z[3])):
        page = torch.tensor([int(c.table[b, p // 64]) for b, p in c.where])
        slot = torch.tensor([p % 64 for _, p in c.where])
        s = sf.cpu().view(E4M3).double()[page, :, slot]                      # [T, 8, 8]
        raw = codes.cpu()[page, :, slot].long()
        v = grid[torch.stack([raw & 15, raw >> 4], -1).flatten(-2)]         # [T, 8, 128]
        off = 2.0 ** -19 * mag
        amax, slack = x.abs().unflatten(-1, (-1, 16)).amax(-1) / 6, off.unflatten(-1, (-1, 16)).amax(-1) / 6 + 2.0 ** -22 * x.abs().unflatten(-1, (-1, 16)).amax(-1)
        nearest = (levels[:, None] - amax.reshape(1, -1)).abs().amin(0).view_as(amax)
        assert ((s - amax).abs() <= nearest + 2 * slack).all()
        y = x / s.repeat_interleave(16, -1)
        near = (grid[:, None] - y.clamp(-6, 6).reshape(1, -1)).abs().amin(0).view_as(y)
        assert ((v - y.clamp(-6, 6)).abs() <= near + 2 * off / s.repeat_interleave(16, -1) + 2.0 ** -22 * y.abs()).all()
    untouched = torch.ones(c.num, 64, dtype=torch.bool)
    untouched[page, slot] = False
    assert (z[0].cpu().permute(0, 2, 1, 3)[untouched] == 0x55).all() and (z[3].cpu().permute(0, 2, 1, 3)[untouched] == 0x55).all()


def test_without_norms_and_positions_nothing_changes():
    """Positions that are the places, with no norm, give the plain append's bits."""
    for cache in (BF16, E4M3):
        c = Case([5, 1, 40], [5, 17, 40], d=128, cache=cache, seed=12)
        got = []
        for positions in (None, torch.tensor([w[1] for w in c.where], dtype=torch.int32, device=DEV)):
            a, kp, vp = c.device(), c.k_pages.to(DEV), c.v_pages.to(DEV)
            q = gqa.gqa_paged_append(**a, k_pages=kp, v_pages=vp, positions=positions, k_scale=0.5 if cache == E4M3 else 1.0)
            got.append((q, kp.view(torch.uint8), vp.view(torch.uint8)))
        assert all(torch.equal(x, y) for x, y in zip(*got))


def test_captured():
    c = Case([1, 1], [5, 9], d=128, seed=13)
    a, kp, vp = c.device(), c.k_pages.to(DEV), c.v_pages.to(DEV)
    w = torch.rand(128, device=DEV)
    want = gqa.gqa_paged_append(**a, k_pages=kp, v_pages=vp, q_norm=w, k_norm=w)
    graph = torch.cuda.CUDAGraph()
    k2, v2 = torch.zeros_like(kp), torch.zeros_like(vp)
    with torch.cuda.graph(graph):
        got = gqa.gqa_paged_append(**a, k_pages=k2, v_pages=v2, q_norm=w, k_norm=w)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    page = c.table[0, 0]
    assert torch.equal(k2[page, :, 4], kp[page, :, 4]) and torch.equal(v2[page, :, 4], vp[page, :, 4])
