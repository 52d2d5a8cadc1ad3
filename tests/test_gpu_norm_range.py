"""GPU: norms of heads whose squares lie at the ends of f32's range, or outside it."""
import pytest
import torch

import gqa_attention_kv_split_gb300 as gqa
from test_gpu_norm_append import check
from test_gpu_paged_append import Case

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


# 2^-131: bf16's subnormal numbers; 2^-84 and 2^-64: squares that are 0 and subnormal; 2^-50: where heads begin to be
# scaled; 2^60 to 2^64: some sums of squares are infinite; 2^120: all
@pytest.mark.parametrize("spread", [2.0 ** e for e in (-131, -100, -84, -64, -53, -50, -47, 50, 60, 61, 62, 64, 120)])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -120, 1e-6])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_heads_of_every_size(spread, eps, d):
    check(Case([4, 3], [4, 9], hq=5, hkv=3, d=d, rot=64, dtype=BF16, seed=d, spread=spread), eps=eps)


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-6, 1e38])
def test_heads_of_different_sizes_in_a_warp(eps):
    """Some rows of a warp are summed once, others twice."""
    c = Case([9, 4], [9, 9], hq=6, hkv=3, d=64, rot=64, dtype=BF16, seed=3)
    for x in (c.q, c.k):
        x *= torch.tensor([2.0 ** -90, 1.0, 2.0 ** 80], dtype=BF16).repeat(x.shape[1] // 3)[None, :, None]
    check(c, eps=float(torch.tensor(eps)))  # (the f32 number that the call takes: 1e-45 is 2^-149)


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (BF16, E4M3)])
def test_heads_of_zeros_stay_zeros(dtype, cache):
    c = Case([3], [3], hq=4, hkv=2, d=128, rot=128, dtype=dtype, cache=cache, seed=4)
    a = c.device()
    a["q"][1, 2] = 0
    a["k"][2, 1] = 0
    kp, vp = c.k_pages.to(DEV), c.v_pages.to(DEV)
    w = torch.ones(128, dtype=dtype, device=DEV)
    got = gqa.gqa_paged_append(**a, k_pages=kp, v_pages=vp, q_norm=w, k_norm=w, norm_eps=0.0)
    assert (got[1, 2] == 0).all() and torch.isfinite(got).all() and (got[0] != 0).any()
    page, slot = int(c.table[0, 2 // c.page]), 2 % c.page
    assert (kp[page, 1, slot].float() == 0).all() and (kp[page, 0, slot].float() != 0).any()
