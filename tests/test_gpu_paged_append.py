"""GPU: gqa_paged_append and nvfp4_paged_append against their plain 64-bit
(NVFP4: bit for bit, 32-bit) forms."""
import math

import pytest
import torch

import gqa_attention_kv_split_gb300 as gqa
import paged_reference as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


def rope_table(n, rot):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


class Case:
    """Inputs on the CPU: q, k, v are slices of one projection's rows; pages hold a sentinel."""

    def __init__(self, q_lens, kv_lens, hq=4, hkv=2, d=64, page=16, rot=None, dtype=torch.bfloat16, cache=None, layout="hnd",
                 seed=0, pad=0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.indptr = [0]
        for n in q_lens:
            self.indptr.append(self.indptr[-1] + n)
        self.total, self.kv_lens, self.page = self.indptr[-1] + pad, list(kv_lens), page
        qkv = (torch.randn(self.total, hq + 2 * hkv, d, generator=g) * spread).to(dtype)
        self.q, self.k, self.v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        mp = max(1, max((n + page - 1) // page for n in kv_lens)) + 1
        self.num = len(kv_lens) * mp
        perm = torch.randperm(self.num, generator=g).to(torch.int32)
        self.table = perm.view(len(kv_lens), mp).clone()
        for b, n in enumerate(kv_lens):  # entries that no token needs are not valid pages
            self.table[b, max(0, (n + page - 1) // page):] = -7
        self.rope = None if rot == 0 else rope_table(max(1, max(kv_lens)), rot or d)
        self.cache = cache or dtype
        shape = (self.num, page, hkv, d) if layout == "nhd" else (self.num, hkv, page, d)
        self.k_pages = torch.full(shape, 3.0, dtype=torch.float32).to(self.cache)
        self.v_pages = torch.full(shape, -3.0, dtype=torch.float32).to(self.cache)
        self.layout, self.where = layout, R.positions(self.total, self.kv_lens, self.indptr)

    def view(self, p):
        return p.permute(0, 2, 1, 3) if self.layout == "nhd" else p

    def device(self):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        wide = torch.cat([self.q, self.k, self.v], 1).to(DEV)
        hq, hkv = self.q.shape[1], self.k.shape[1]
        return dict(q=wide[:, :hq], k=wide[:, hq:hq + hkv], v=wide[:, hq + hkv:], block_table=self.table.to(DEV),
                    kv_lens=i32(self.kv_lens), qo_indptr=i32(self.indptr), rope=None if self.rope is None else self.rope.to(DEV))


def bound(x, mag, dtype, inv=1.0):
    """Half a step of the stored type around the exact value, and three f32 roundings of the terms."""
    slack = 2.0 ** -22 * mag * inv
    if dtype == torch.float8_e4m3fn:
        return torch.maximum(2.0 ** -4 * x.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64)) * (1 + 2.0 ** -10) + slack
    f = torch.finfo(dtype)
    return f.eps / 2 * x.abs() * (1 + f.eps) + slack + f.smallest_normal * f.eps


def check(c: Case, interleaved=False, k_scale=1.0, v_scale=1.0, one_each=False, **kw):
    a = c.device()
    kp, vp = c.k_pages.to(DEV), c.v_pages.to(DEV)
    if one_each:
        a["qo_indptr"] = None
    q_out = torch.full((c.total,) + c.q.shape[1:], 7.0, dtype=c.q.dtype, device=DEV)
    got = gqa.gqa_paged_append(**a, k_pages=c.view(kp), v_pages=c.view(vp), interleaved=interleaved, k_scale=k_scale, v_scale=v_scale,
                               q_out=q_out, **kw)
    torch.cuda.synchronize()
    assert got is q_out
    mag = lambda x: R.rotated(x.abs(), None if c.rope is None else c.rope.abs() * torch.cat([torch.ones(c.rope.shape[1] // 2), -torch.ones(c.rope.shape[1] // 2)]),
                              c.where, interleaved).abs() + x.abs().double()
    live = torch.tensor([w is not None and w[1] >= 0 for w in c.where])
    want_q = R.rotated(c.q, c.rope, c.where, interleaved)
    err = (got.cpu().double() - want_q)[live].abs()
    assert (err <= bound(want_q, 2 * mag(c.q), c.q.dtype)[live]).all(), f"q: {float(err.max())}"
    assert (got.cpu()[~live] == 7.0).all()
    for name, x, pages, scale, dev in (("k", R.rotated(c.k, c.rope, c.where, interleaved), c.k_pages, k_scale, kp),
                                       ("v", c.v.double(), c.v_pages, v_scale, vp)):
        x = x / scale
        if c.cache == torch.float8_e4m3fn:
            x = x.clamp(-448, 448)
        want, tol = pages.double().clone(), torch.zeros(pages.shape, dtype=torch.float64)
        R.place(c.view(want), x, c.where, c.table, c.page)
        m = 2 * mag(c.k) if name == "k" else c.v.double().abs()
        R.place(c.view(tol), bound(x, m, c.cache, 1 / scale), c.where, c.table, c.page)
        e = (dev.cpu().double() - want).abs()
        assert (e <= tol).all(), f"{name}: {float(e.max())}"  # untouched slots: exactly as they were


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (64, 16, False), (64, 48, True), (128, 128, False), (128, 64, True),
                                         (128, 0, False), (256, 256, False), (256, 80, False), (256, 256, True)])
def test_append_matches_plain_form(dtype, d, rot, inter):
    check(Case([5, 1, 40], [5, 17, 40], d=d, rot=rot, dtype=dtype, seed=d + rot), interleaved=inter)


@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("hq,hkv,page", [(1, 1, 16), (5, 1, 32), (28, 4, 64), (12, 12, 1), (7, 7, 5), (40, 2, 128)])
def test_append_head_counts_pages_and_orders(layout, hq, hkv, page):
    check(Case([3, 9], [130, 9], hq=hq, hkv=hkv, page=page, layout=layout, seed=hq))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_append_to_e4m3_pages(dtype, d):
    c = Case([33, 2], [64, 9], d=d, dtype=dtype, cache=torch.float8_e4m3fn, layout="nhd", seed=5, spread=3.0)
    check(c, k_scale=0.03, v_scale=2.5)
    check(c, k_scale=0.001, v_scale=1.0)  # saturates


def test_append_one_token_each_and_long_tables():
    n = 300
    check(Case([1] * n, [1 + 37 * i % 501 for i in range(n)], seed=6), one_each=True)
    check(Case([1] * n, [1 + 37 * i % 501 for i in range(n)], seed=6))


def test_append_many_sequences_with_empty_ones():
    """Searches of more than 32 (and 1024) offsets, runs of empty sequences, a first and a last one empty."""
    q = [0] + [i % 3 for i in range(1100)] + [0, 4, 0]
    check(Case(q, [n + i % 20 for i, n in enumerate(q)], hq=2, hkv=1, seed=7))


def test_append_skips_padding_and_inactive_sequences():
    c = Case([2, 1, 3], [2, 0, 1], seed=8, pad=5)  # positions -1 (inactive) and -2, -1, 0
    assert sum(w is None for w in c.where) == 5
    check(c)
    assert gqa.gqa_check_device_errors(0) == 0


def test_append_block_of_tokens_per_block():
    """Enough tokens that a block takes eight, the last one fewer."""
    check(Case([4999], [4999], hq=2, hkv=1, seed=9))


def test_append_in_place_and_without_q():
    c = Case([20, 3], [20, 40], d=128, seed=10)
    a = c.device()
    p = [c.k_pages.to(DEV) for _ in range(3)]
    out = gqa.gqa_paged_append(**a, k_pages=p[0], v_pages=c.v_pages.to(DEV))
    b = c.device()
    same = gqa.gqa_paged_append(**b, k_pages=p[1], v_pages=c.v_pages.to(DEV), q_out=b["q"])
    assert same is b["q"] and torch.equal(same, out) and torch.equal(p[0], p[1])
    a["q"] = None
    assert gqa.gqa_paged_append(**a, k_pages=p[2], v_pages=c.v_pages.to(DEV)) is None
    assert torch.equal(p[0], p[2])


def test_append_broadcast_values():
    """An expanded input (stride 0) is read like any other."""
    c = Case([4], [4], hkv=2, seed=11)
    a = c.device()
    one = a["v"][:, :1].contiguous()
    p, r = [c.v_pages.to(DEV) for _ in range(2)], c.k_pages.to(DEV)
    gqa.gqa_paged_append(**{**a, "v": one.expand(-1, 2, -1)}, k_pages=r, v_pages=p[0])
    gqa.gqa_paged_append(**{**a, "v": one.repeat(1, 2, 1)}, k_pages=r, v_pages=p[1])
    assert torch.equal(p[0], p[1])


@pytest.mark.parametrize("what", ["page", "low page", "table", "rope", "offsets", "first offset"])
def test_append_flags_bad_metadata_and_leaves_the_rest(what):
    c = Case([3, 2], [20, 18], seed=12)
    a = c.device()
    bad = {0, 1, 2}
    if what == "page":
        a["block_table"][0, 1] = c.num
    elif what == "low page":
        a["block_table"][0, 1] = -1
    elif what == "table":
        a["kv_lens"][0] = 16 * c.table.shape[1] + 3
    elif what == "rope":
        a["rope"] = a["rope"][:19].contiguous()
        bad = {2}
    elif what == "offsets":
        a["qo_indptr"][2] = 50  # 50 new tokens end behind the inputs
        a["kv_lens"][1] = 18 + 45
        a["block_table"][1, 1] = a["block_table"][1, 0]
        bad = set()
    else:
        a["qo_indptr"][0] = 3
    kp, vp = c.k_pages.to(DEV), c.v_pages.to(DEV)
    q_out = torch.full((c.total,) + c.q.shape[1:], 7.0, dtype=c.q.dtype, device=DEV)
    gqa.gqa_paged_append(**a, k_pages=kp, v_pages=vp, q_out=q_out)
    bit = 4 if "offset" in what else 2
    assert gqa.gqa_check_device_errors(0) & bit
    left = (q_out.cpu() == 7.0).flatten(1).all(1)
    assert {t for t in range(c.total) if left[t]} == bad
    if what == "offsets":
        return
    want = c.v_pages.clone()
    R.place(want, c.v, [w if t not in bad else None for t, w in enumerate(c.where)], c.table, c.page)
    assert torch.equal(vp.cpu(), want)


# ---- NVFP4 ---------------------------------------------------------------------

def nvfp4_check(q_lens, kv_lens, *, rot=128, inter=False, dtype=torch.bfloat16, seed=0, q_scale=0.05, pad=0, edit=None, indptr=True):
    c = Case(q_lens, kv_lens, hq=32, hkv=8, d=128, page=64, rot=rot, dtype=dtype, seed=seed, pad=pad)
    if edit:
        edit(c)
    a = c.device()
    if not indptr:
        a["qo_indptr"] = None
    codes = [torch.full((c.num, 8, 64, 64), 0x55, dtype=torch.uint8, device=DEV) for _ in range(2)]
    sf = [torch.full((c.num, 8, 64, 8), 0x2A, dtype=torch.uint8, device=DEV) for _ in range(2)]
    q_out = torch.full((c.total, 32, 128), 0x11, dtype=torch.uint8, device=DEV)
    got = gqa.nvfp4_paged_append(a["q"], a["k"], a["v"], codes[0], sf[0], codes[1], sf[1], a["block_table"], a["qo_indptr"], a["kv_lens"],
                                 rope=a["rope"], interleaved=inter, q_scale=q_scale, q_out=q_out)
    torch.cuda.synchronize()
    live = torch.tensor([w is not None and w[1] >= 0 for w in c.where])
    f32 = torch.float32
    inv = torch.tensor(1.0) / torch.tensor(q_scale, dtype=f32)
    want_q = (R.rotated(c.q, c.rope, c.where, inter, f32) * inv).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    gq = got.cpu().view(torch.float8_e4m3fn).float()
    assert torch.equal(gq[live].nan_to_num(999.0), want_q[live].nan_to_num(999.0))
    assert (got.cpu()[~live] == 0x11).all()
    for i, x in enumerate((R.rotated(c.k, c.rope, c.where, inter, f32), c.v.float())):
        val, scale = R.nvfp4_quantise(x)
        want = R.e2m1_decode(torch.full((c.num, 8, 64, 64), 0x55, dtype=torch.uint8))
        want_sf = torch.full((c.num, 8, 64, 8), 0x2A, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
        R.place(want, val, c.where, c.table, 64)
        R.place(want_sf, scale, c.where, c.table, 64)
        assert torch.equal(sf[i].cpu().view(torch.float8_e4m3fn).float().nan_to_num(999.0), want_sf.nan_to_num(999.0)), "kv"[i]
        assert torch.equal(R.e2m1_decode(codes[i].cpu()), want), "kv"[i]
    return c


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rot,inter", [(128, False), (128, True), (64, False), (96, False), (32, True), (0, False)])
def test_nvfp4_append_bit_for_bit(dtype, rot, inter):
    nvfp4_check([5, 70, 1], [5, 70, 130], rot=rot, inter=inter, dtype=dtype, seed=rot)


def test_nvfp4_append_single_tokens_and_padding():
    nvfp4_check([1] * 9, [1, 64, 65, 3, 128, 0, 77, 2, 500], seed=3, indptr=False)
    nvfp4_check([2, 0, 3], [2, 9, 1], seed=4, pad=3)


def test_nvfp4_append_values_that_round():
    """Zero blocks, blocks whose scale underflows to 0 or saturates, exact ties, infinities and NaN."""
    def edit(c):
        v, k = c.v, c.k
        v[0, 0] = 0
        v[0, 1, :16] = 2.0 ** -9      # amax / 6 below half the smallest scale
        v[0, 2, :16] = 30000.0        # scale saturates at 448, codes at 6
        v[0, 3, :16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6])
        v[1, 0, 3] = math.inf
        v[1, 1, 5] = -math.inf
        v[1, 2, 7] = math.nan
        k[1, 3, 20] = math.nan
    nvfp4_check([3], [3], rot=32, seed=5, edit=edit)


def test_nvfp4_append_then_context_attention_reads_it():
    """The written pages are what nvfp4_paged_ctx_attn takes: the same as pages of the existing encoder."""
    import gqa_workloads as W
    c = Case([70, 33], [70, 100], hq=32, hkv=8, d=128, page=64, rot=0, seed=6)
    x = W.make_ctx_inputs([70, 33], [70, 100], seed=6, device="cpu")
    a = c.device()
    kf, ks, vf, vs = (t.to(DEV) for t in (x.k_fp4, x.k_sf, x.v_fp4, x.v_sf))
    table = x.block_table.to(DEV)
    q8 = gqa.nvfp4_paged_append(a["q"], a["k"], a["v"], kf, ks, vf, vs, table, a["qo_indptr"], a["kv_lens"], q_scale=0.01)
    mine = [t.cpu() for t in (kf, ks, vf, vs)]
    for t, src in ((x.k_fp4, x.k_sf), c.k), ((x.v_fp4, x.v_sf), c.v):
        codes, sf = W.quantize_nvfp4(src.float())
        R.place(t[0], codes, c.where, x.block_table, 64)
        R.place(t[1], sf, c.where, x.block_table, 64)
    assert torch.equal(mine[1], x.k_sf) and torch.equal(mine[3], x.v_sf)
    assert torch.equal(R.e2m1_decode(mine[0]), R.e2m1_decode(x.k_fp4)) and torch.equal(R.e2m1_decode(mine[2]), R.e2m1_decode(x.v_fp4))
    run = lambda *p: gqa.nvfp4_paged_ctx_attn(q8, *p, table, a["qo_indptr"], a["kv_lens"], q_scale=0.01, out_scale=2.0 ** -4)
    assert torch.equal(run(kf, ks, vf, vs), run(*(t.to(DEV) for t in (x.k_fp4, x.k_sf, x.v_fp4, x.v_sf))))


def _spread(values):
    """Each f32 value, its two neighbours, and theirs."""
    v = torch.tensor(values, dtype=torch.float32)
    bits = v.view(torch.int32)
    return torch.stack([(bits + i).view(torch.float32) for i in (-2, -1, 0, 1, 2)], -1)


def _quantise_through_keys(rows):
    """Codes' values and scales that the GPU gives rows [T, 64] of f32 (T <= 64 k): keys of ones turned by them."""
    T = rows.shape[0]
    rope = torch.cat([rows, torch.zeros(T, 64)], 1).to(DEV)
    k = torch.ones(T, 8, 128, dtype=torch.bfloat16, device=DEV)
    pages = (T + 63) // 64
    z = lambda w: torch.zeros(pages, 8, 64, w, dtype=torch.uint8, device=DEV)
    kf, ks, vf, vs = z(64), z(8), z(64), z(8)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    gqa.nvfp4_paged_append(None, k, k, kf, ks, vf, vs, torch.arange(pages, dtype=torch.int32, device=DEV)[None], i32(0, T), i32(T), rope=rope)
    val = R.e2m1_decode(kf.cpu()).permute(0, 2, 1, 3).flatten(0, 1)[:T, 0, :64]
    sf = ks.cpu().view(torch.float8_e4m3fn).float().permute(0, 2, 1, 3).flatten(0, 1)[:T, 0, :4]
    return val, sf


def test_nvfp4_codes_at_every_border_of_every_scale():
    """x / sf next to each border between two codes (and on it), for all 126 scales: what f32 division and rounding give."""
    scales = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    rows = []
    for s in scales.tolist():
        near = torch.cat([_spread([t * s for t in (.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0)]).flatten(), torch.tensor([s / 3, s * 5.9, s * 1e-9])])
        row = torch.zeros(64)
        row[0::16] = 6 * s  # gives every block the scale s
        body = torch.tensor([i for i in range(64) if i % 16])
        row[body[:len(near)]] = near * torch.where(torch.arange(len(near)) % 2 == 0, 1.0, -1.0)
        rows.append(row)
    rows = torch.stack(rows)
    val, sf = _quantise_through_keys(rows)
    want, want_sf = R.nvfp4_quantise(rows)
    assert torch.equal(sf, want_sf) and torch.equal(sf, scales[:, None].expand(-1, 4))
    assert torch.equal(val, want)


def test_nvfp4_scales_at_every_border():
    """amax / 6 next to each border between two scales: what f32 division and rounding give."""
    e = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    near = _spread([6 * (a + b) / 2 for a, b in zip(e[:-1].tolist(), e[1:].tolist())] + [448 * 6.0, 464 * 6.0, 3e38]).flatten()
    near = near[torch.isfinite(near)]
    near = torch.cat([near, torch.full((-len(near) % 4,), 1.0)]).view(-1, 4)
    rows = torch.zeros(len(near), 64)
    rows[:, 5::16] = near
    val, sf = _quantise_through_keys(rows)
    want, want_sf = R.nvfp4_quantise(rows)
    assert torch.equal(sf, want_sf) and torch.equal(val, want)
