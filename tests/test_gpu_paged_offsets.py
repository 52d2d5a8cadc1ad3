"""GPU: offsets that do not run from 0 upwards are flagged, whichever token they concern."""
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


def run(indptr, total, nvfp4=False):
    """Appends `total` tokens under these offsets and returns the error word."""
    B = len(indptr) - 1
    hq, hkv, d, page = (32, 8, 128, 64) if nvfp4 else (4, 2, 64, 64)
    x = torch.randn(total, hq + 2 * hkv, d, device=DEV).bfloat16()
    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None]
    lens = torch.full((B,), page, dtype=torch.int32, device=DEV)
    start = torch.tensor(indptr, dtype=torch.int32, device=DEV)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if nvfp4:
        z = [torch.zeros(B, hkv, page, w, dtype=torch.uint8, device=DEV) for w in (d // 2, d // 16) * 2]
        gqa.nvfp4_paged_append(q, k, v, *z, table, start, lens)
    else:
        p = [torch.zeros(B, hkv, page, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        gqa.gqa_paged_append(q, k, v, *p, table, lens, qo_indptr=start)
    return gqa.gqa_check_device_errors(0)


@pytest.mark.parametrize("nvfp4", [False, True])
@pytest.mark.parametrize("indptr,total", [([0, 5, 3], 5), ([0, 4, 2, 5], 5), ([-1, 2, 5], 5), ([2, 5], 5), ([0, 5, 5, 4, 5], 6),
                                          ([0] + [9] * 1500 + [8, 9], 9)])
def test_offsets_that_go_down_are_flagged(indptr, total, nvfp4):
    assert run(indptr, total, nvfp4) == 4


@pytest.mark.parametrize("indptr,total", [([0, 0, 0, 5], 5), ([0, 5, 5], 9), ([0, 0], 3), ([0] + [9] * 1500, 9)])
def test_offsets_of_empty_sequences_and_padding_are_not(indptr, total):
    assert run(indptr, total) == 0
