"""GPU: gqa_paged_tree_attn over offsets that go back again and again, so that sequences in order share rows and have
more of them together than there are."""
import pytest
import torch

import gqa_attention_kv_split_gb300 as gqa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("short", [128, 160, 256])
def test_sequences_over_the_same_rows(short):
    """A capacity and a number of rows for which no unit would have to be split, most of them gone through twice: the two
    sequences around offsets that fall have the same cached tokens before their first row, and so the same rows."""
    g = torch.Generator().manual_seed(short)
    n, before = 480, 20
    q = torch.randn(n, 32, 128, generator=g).half().to(DEV)
    k, v = (torch.randn(8, 8, 64, 128, generator=g).half().to(DEV) for _ in range(2))
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(1, 8)
    lse = torch.full((n, 32), 9.0, device=DEV)
    want = gqa.gqa_paged_tree_attn(q, k, v, table, i32([0, n]), i32([before + n]), lse=lse)
    out, got_lse = torch.full_like(q, 5.0), torch.full_like(lse, 9.0)
    gqa.gqa_paged_tree_attn(q, k, v, table.repeat(3, 1), i32([0, short, 0, n]), i32([before + short, 7, before + n]), out=out, lse=got_lse)
    assert gqa.gqa_check_device_errors(0) == 4
    assert torch.equal(out, want) and torch.equal(got_lse, lse)


def test_more_work_than_shares_can_count():
    """2048 times the same 16384 tokens of 64 heads over 3.2 million cached ones: a block's share would pass 31 bits.
    (The producers are starved, so that a kernel that began with it would give up.)"""
    n, batch, cols = 16384, 4096, 12500
    q = torch.zeros(n, 64, 64, dtype=torch.float16, device=DEV)
    k = torch.zeros(1, 1, 256, 64, dtype=torch.float16, device=DEV)
    table = torch.zeros(batch, cols, dtype=torch.int32, device=DEV)
    assert batch // 2 * (n * 64 // 128) * (cols * 256 // 128 + 5) // 152 > 2 ** 31
    out = torch.full_like(q, 5.0)
    gqa.gqa_debug_starve_producers(True)
    try:
        gqa.gqa_paged_tree_attn(q, k, k, table, i32([0, n] * (batch // 2) + [0]), i32([cols * 256] * batch), out=out)
        assert gqa.gqa_check_device_errors(0) == 4
    finally:
        gqa.gqa_debug_starve_producers(False)
    assert (out == 5.0).all()
