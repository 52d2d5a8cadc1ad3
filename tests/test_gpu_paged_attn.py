"""GPU: gqa_paged_attn against the plain 64-bit form, within the bound that
paged_reference.check_attention derives."""
import math

import pytest
import torch

import gqa_attention_kv_split_gb300 as gqa
import paged_reference as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


def make(lens, hq=4, hkv=2, d=128, page=16, dtype=F16, cache=None, layout="hnd", seed=0, spread=1.0, poison=True, window=0):
    """q, pages, table, lens on the GPU; slots that no token sees hold NaN, table entries that none needs -1."""
    g = torch.Generator().manual_seed(seed)
    cache = cache or dtype
    B, mp = len(lens), max(1, max((max(n, 0) + page - 1) // page for n in lens)) + 1
    num = B * mp
    q = (torch.randn(B, hq, d, generator=g) * spread).to(dtype)
    table = torch.randperm(num, generator=g).to(torch.int32).view(B, mp)
    pages = []
    for _ in range(2):
        x = torch.randn(num, hkv, page, d, generator=g)
        x = (x * 16).clamp(-448, 448).to(cache) if cache == E4M3 else x.to(cache)
        pages.append(x)
    if poison:
        seen = torch.zeros(num, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for t in range(max(0, n - window) if window else 0, max(n, 0)):
                seen[table[b, t // page], t % page] = True
            used = torch.arange(mp)
            lo = (max(0, n - window) if window else 0) // page
            table[b][(used >= (max(n, 0) + page - 1) // page) | (used < lo)] = -1
        for x in pages:
            raw = x.view(torch.uint8) if cache == E4M3 else x
            raw.permute(0, 2, 1, 3)[~seen] = 0x7F if cache == E4M3 else math.nan
    k, v = (x.permute(0, 2, 1, 3).contiguous().to(DEV).permute(0, 2, 1, 3) if layout == "nhd" else x.to(DEV) for x in pages)
    return q.to(DEV), k, v, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def clean(k, v):
    return [torch.nan_to_num(x.float(), nan=0.0).to(x.dtype) for x in (k.cpu(), v.cpu())]


def check(x, **kw):
    q, k, v, table, lens = x
    lse = torch.full(q.shape[:2], 9.0, device=DEV)
    out = gqa.gqa_paged_attn(q, k, v, table, lens, lse=lse, **kw)
    torch.cuda.synchronize()
    kc, vc = clean(k, v)
    R.check_attention(out, lse, q, kc, vc, table.clamp(min=0), lens, **kw)
    return out, lse


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 0, 128, 200, 700]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)])
def test_matches_plain_form(dtype, cache, d):
    check(make(LENS, d=d, dtype=dtype, cache=cache, seed=d))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (4, 1), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 2), (32, 8), (12, 12)])
@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_groups_of_every_size(hq, hkv, cache):
    check(make([33, 150, 1, 0], hq=hq, hkv=hkv, d=64, dtype=BF16, cache=cache, seed=hq))
    check(make([90], hq=hq, hkv=hkv, d=128, dtype=BF16, cache=cache, seed=hq))


@pytest.mark.parametrize("group", [9, 16])
@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (BF16, E4M3)])
def test_two_blocks_of_heads_at_head_dim_256(dtype, cache, group):
    check(make([300, 31], hq=group, hkv=1, d=256, dtype=dtype, cache=cache, seed=group))


@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("cache,d", [(F16, 128), (E4M3, 64), (E4M3, 256), (F16, 256)])
def test_pages_and_orders(layout, page, cache, d):
    check(make([1, 77, 300, 513], d=d, page=page, cache=cache, layout=layout, seed=page))


@pytest.mark.parametrize("window", [1, 2, 16, 17, 63, 64, 65, 100, 129, 5000])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_window(window, d):
    """Keys before the window are not read: their slots hold NaN and their table entries are -1."""
    check(make([0, 1, 16, 64, 65, 100, 400], d=d, window=window, seed=window), window=window)


@pytest.mark.parametrize("window", [0, 1, 127, 128, 129])
@pytest.mark.parametrize("cache,d", [(F16, 256), (F16, 128), (F16, 64), (E4M3, 64)])
def test_tile_borders(window, cache, d):
    """Lengths and windows around the tiles' 32, 64 and 128 tokens, in the smallest and the largest pages."""
    lens = [31, 32, 33, 127, 128, 129, 255, 256, 257, 385]
    for page in (16, 256):
        check(make(lens, d=d, page=page, cache=cache, window=window, seed=window), window=window)


@pytest.mark.parametrize("softcap", [0.5, 30.0])
@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, E4M3)])
def test_softcap(softcap, dtype, cache):
    check(make([300, 5], dtype=dtype, cache=cache, spread=4.0, seed=3), softcap=softcap)


def test_scales():
    x = make([100, 300], cache=E4M3, dtype=BF16, seed=4)
    check(x, q_scale=0.7, k_scale=1 / 16, v_scale=1 / 64)
    check(x, q_scale=-1.0, k_scale=1 / 16)
    check(make([100], seed=4), q_scale=0.0)


@pytest.mark.parametrize("scale", [2.0 ** -100, 1.0, 2.0 ** 100])
def test_bf16_queries_of_any_size_over_e4m3_pages(scale):
    """A bf16 query row is brought into f16's range by a power of two."""
    q, k, v, table, lens = make([80, 33], cache=E4M3, dtype=BF16, seed=5)
    q[:, 0] = 0
    check((q * scale, k, v, table, lens), q_scale=1.0 / scale / 16)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_sharp_and_rising_scores(dtype):
    """Scores of hundreds that keep rising along the sequence: every tile moves the maximum."""
    q, k, v, table, lens = make([700], hq=2, hkv=1, dtype=dtype, seed=6)
    up = torch.arange(k.shape[2] * table.shape[1], device=DEV).float() / 20
    for t in range(700):
        pg, s = int(table[0, t // 16]), t % 16
        k[pg, 0, s] = (up[t] * q[0, 0].float() / q[0, 0].float().norm()).to(dtype)
    check((q, k, v, table, lens))


def test_many_small_weights_are_kept():
    """One large weight and 30000 of 2^-17 of it: together a fifth of the sum, in f16 pages."""
    n = 30000
    q, k, v, table, lens = make([n], hq=1, hkv=1, d=64, page=64, poison=False, seed=7)
    q.zero_()
    q[..., 0] = 1.0
    k.zero_()
    pg = int(table[0, 0])
    k[pg, 0, 0, 0] = 17 * math.log(2) * 8.0
    check((q, k, v, table, lens))


@pytest.mark.parametrize("B,hq,hkv,d", [(1, 8, 8, 128), (1, 8, 1, 64), (2, 16, 8, 256), (3, 64, 4, 128)])
def test_split_over_long_sequences(B, hq, hkv, d):
    """Few sequences: each unit lies in many blocks' shares, and in two blocks' pieces at least."""
    check(make([5000 + 777 * i for i in range(B)], hq=hq, hkv=hkv, d=d, page=64, poison=False, dtype=BF16, seed=8))


@pytest.mark.parametrize("hq,hkv", [(5, 5), (6, 6), (12, 12), (16, 16), (24, 24), (152, 152), (20, 2), (72, 3), (160, 8)])
@pytest.mark.parametrize("lens", [(3000, 0, 1, 700, 64, 65), (130,) * 9, (0, 40, 0, 2100)])
def test_blocks_that_share_sequences(hq, hkv, lens):
    """Blocks that read the same tokens for 1, 2, 4 or 8 units of a sequence, once or in several turns."""
    check(make(lens, hq=hq, hkv=hkv, d=64, page=32, seed=hq))
    check(make(lens, hq=hq, hkv=hkv, d=128, page=16, layout="nhd", dtype=BF16, cache=E4M3, seed=hkv))


def test_more_sequences_than_threads():
    """Several sequences a thread in the division of the work, empty ones among them."""
    lens = [(i * 37) % 40 if i % 5 else 0 for i in range(701)]
    check(make(lens, hq=2, hkv=1, d=64, page=16, seed=9))


def test_all_empty():
    out, lse = check(make([0, -3, 0], seed=10))
    assert torch.count_nonzero(out) == 0 and torch.isinf(lse).all()


def test_lengths_are_clamped_to_the_table():
    q, k, v, table, lens = make([64, 64], page=16, poison=False, seed=11)
    cap = table.shape[1] * 16
    a = gqa.gqa_paged_attn(q, k, v, table, torch.tensor([cap + 999, -1], dtype=torch.int32, device=DEV))
    b = gqa.gqa_paged_attn(q, k, v, table, torch.tensor([cap, 0], dtype=torch.int32, device=DEV))
    assert torch.equal(a, b)


def test_strided_queries_and_no_lse():
    q, k, v, table, lens = make([70, 9], seed=12)
    wide = torch.randn(2, 7, 128, device=DEV).half()
    wide[:, 1:5] = q
    assert torch.equal(gqa.gqa_paged_attn(wide[:, 1:5], k, v, table, lens), gqa.gqa_paged_attn(q, k, v, table, lens))


def test_stacked_cache_as_views():
    """K and V of one allocation [num_pages, 2, page, heads, d], as other engines keep it."""
    q, k, v, table, lens = make([70, 300], seed=13, poison=False)
    both = torch.stack([k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)], 1).contiguous()
    a = gqa.gqa_paged_attn(q, both[:, 0].permute(0, 2, 1, 3), both[:, 1].permute(0, 2, 1, 3), table, lens)
    assert torch.equal(a, gqa.gqa_paged_attn(q, k, v, table, lens))


def test_repeated_calls_give_the_same_bits():
    x = make([3000, 10, 977, 1], hq=16, hkv=2, poison=False, seed=14)
    a = gqa.gqa_paged_attn(*x)
    for _ in range(3):
        assert torch.equal(a, gqa.gqa_paged_attn(*x))


def test_bad_page_is_flagged_and_not_read():
    q, k, v, table, lens = make([100], seed=15, poison=False)
    table[0, 2] = 1 << 20
    a = gqa.gqa_paged_attn(q, k, v, table, lens)
    assert gqa.gqa_check_device_errors(0) & 2
    table[0, 2] = 0
    assert torch.equal(a, gqa.gqa_paged_attn(q, k, v, table, lens))
    assert gqa.gqa_check_device_errors(0) == 0


def test_agrees_with_the_other_decodes():
    """The same pages through gqa_decode_paged."""
    import gqa_workloads as W
    p = W.page_decode_inputs(W.make_decode_inputs(3, 2048, [2048, 1, 700], seed=84), seed=84)
    a = [t.to(DEV) for t in (p.q, p.k_pages, p.v_pages, p.block_table, p.seq_lens)]
    out, _ = check(a)
    assert (out.float() - gqa.gqa_decode_paged(*a).float()).abs().max() <= 2.0 ** -10


def test_expired_waits_are_reported():
    x = make([100, 300], seed=16, poison=False)
    good = gqa.gqa_paged_attn(*x)
    gqa.gqa_debug_starve_producers(True)
    try:
        gqa.gqa_paged_attn(*x)
        assert gqa.gqa_check_device_errors(0) & 1
    finally:
        gqa.gqa_debug_starve_producers(False)
    assert torch.equal(good, gqa.gqa_paged_attn(*x))
    assert gqa.gqa_check_device_errors(0) == 0


def test_scales_out_of_range_are_refused():
    x = make([20], seed=17, poison=False)
    with pytest.raises(gqa.GqaError, match="out of range"):
        gqa.gqa_paged_attn(*x, q_scale=3e38, k_scale=1e30)
    with pytest.raises(gqa.GqaError, match="out of range"):
        gqa.gqa_paged_attn(*x, q_scale=1e20, softcap=1e-30)
