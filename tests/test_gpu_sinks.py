"""GPU: gqa_paged_attn with a window and sinks against the plain 64-bit form, within the bound that
draft_reference.check_attention derives."""
import math

import pytest
import torch

import draft_reference as DR
import gqa_attention_kv_split_gb300 as gqa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


def make(lens, visible, hq=4, hkv=2, d=128, page=16, dtype=F16, cache=None, layout="hnd", seed=0, rows=None, spread=1.0):
    """q (a row each, or `rows` of a sequence), pages, table, lens on the GPU; slots that no token sees hold NaN,
    pages without a visible one are not in the table."""
    g = torch.Generator().manual_seed(seed)
    cache = cache or dtype
    B, mp = len(lens), max(1, max((max(n, 0) + page - 1) // page for n in lens)) + 1
    num = B * mp
    q = (torch.randn(len(visible), hq, d, generator=g) * spread).to(dtype)
    full = torch.randperm(num, generator=g).to(torch.int32).view(B, mp)
    seq = rows or list(range(B))
    seen = torch.zeros(num, page, dtype=torch.bool)
    used = torch.zeros(B, mp, dtype=torch.bool)
    for b, places in zip(seq, visible):
        if places:
            at = torch.tensor(places)
            seen[full[b].long()[at // page], at % page] = True
            used[b, at // page] = True
    table = torch.where(used, full, -1).to(torch.int32)
    pages = []
    for _ in range(2):
        x = torch.randn(num, hkv, page, d, generator=g)
        x = (x * 16).clamp(-448, 448).to(cache) if cache == E4M3 else x.to(cache)
        raw = x.view(torch.uint8) if cache == E4M3 else x
        raw.permute(0, 2, 1, 3)[~seen] = 0x7F if cache == E4M3 else math.nan
        pages.append(x)
    k, v = (x.permute(0, 2, 1, 3).contiguous().to(DEV).permute(0, 2, 1, 3) if layout == "nhd" else x.to(DEV) for x in pages)
    return q.to(DEV), k, v, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), seq


def clean(k, v):
    return [torch.nan_to_num(x.float(), nan=0.0).to(x.dtype) for x in (k.cpu(), v.cpu())]


def check(lens, window, sinks, softcap=0.0, scales=(1.0, 1.0), **kw):
    visible = [DR.visible_one(n, window, sinks) for n in lens]
    q, k, v, table, d_lens, seq = make(lens, visible, **kw)
    lse = torch.full(q.shape[:2], 9.0, device=DEV)
    out = gqa.gqa_paged_attn(q, k, v, table, d_lens, lse=lse, window=window, sinks=sinks, softcap=softcap, k_scale=scales[0], v_scale=scales[1])
    torch.cuda.synchronize()
    DR.check_attention(out, lse, q, *clean(k, v), table.cpu().clamp(min=0), visible, softcap=softcap, k_scale=scales[0], v_scale=scales[1])
    return out, lse


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 0, 128, 200, 700]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)])
def test_matches_plain_form(dtype, cache, d):
    check(LENS, 48, 4, d=d, dtype=dtype, cache=cache, seed=d)
    check(LENS, 5, 70, d=d, dtype=dtype, cache=cache, seed=d + 1, layout="nhd")


@pytest.mark.parametrize("window", [1, 15, 16, 31, 64, 129, 690, 5000])
@pytest.mark.parametrize("sinks", [1, 16, 33, 64, 128, 300, 698, 9999])
def test_windows_and_sinks(window, sinks):
    """Sinks that end in the window's tile, before it, within it and behind it."""
    check(LENS, window, sinks, d=64, seed=window)
    check([700, 900], window, sinks, d=128, page=64, cache=E4M3, scales=(0.1, 0.2), seed=sinks)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (7, 1), (17, 1), (40, 2), (12, 12)])
def test_pages_and_groups(page, hq, hkv):
    check([600, 33, 1000, 0], 100, 20, page=page, hq=hq, hkv=hkv, dtype=BF16, seed=page)


def test_caps():
    check([600, 100], 64, 4, softcap=20.0, dtype=BF16, seed=2, spread=4.0)


@pytest.mark.parametrize("hkv", [1, 8])
def test_long_sequences_split_over_blocks(hkv):
    """Tiles of the sinks and of the window in several blocks' shares."""
    check([40000, 9000, 20000], 7000, 3000, hq=4 * hkv, hkv=hkv, page=64, dtype=BF16, seed=5)
    check([60000], 30000, 4, hq=8 * hkv, hkv=hkv, page=64, cache=E4M3, seed=6)


def test_sinks_of_nothing():
    """0 sinks, and sinks without a window, are the calls without them, to the bit."""
    q, k, v, table, lens, _ = make([300, 50], [list(range(300)), list(range(50))], seed=7)
    for kw in (dict(window=0), dict(window=100)):
        a = gqa.gqa_paged_attn(q, k, v, table, lens, **kw)
        assert torch.equal(a, gqa.gqa_paged_attn(q, k, v, table, lens, sinks=0, **kw))
    assert torch.equal(gqa.gqa_paged_attn(q, k, v, table, lens), gqa.gqa_paged_attn(q, k, v, table, lens, sinks=30))


def test_captured_call_follows_the_lengths():
    visible = [list(range(900)), list(range(500))]
    q, k, v, table, lens, _ = make([900, 500], visible, dtype=BF16, seed=8)
    now = lens.clone()
    lse = torch.zeros(2, 4, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gqa.gqa_paged_attn(q, k, v, table, now, lse=lse, window=64, sinks=4)
    for n in ([900, 3], [70, 500], [0, 68]):
        now.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        DR.check_attention(out, lse, q, *clean(k, v), table.cpu(), [DR.visible_one(x, 64, 4) for x in n])


def test_bad_pages_are_flagged():
    q, k, v, table, lens, _ = make([300], [list(range(300))], seed=9)
    table[0, 0] = 10 ** 6
    gqa.gqa_paged_attn(q, k, v, table, lens, window=16, sinks=0)
    assert gqa.gqa_check_device_errors(0) == 0
    gqa.gqa_paged_attn(q, k, v, table, lens, window=16, sinks=4)
    assert gqa.gqa_check_device_errors(0) == 2
