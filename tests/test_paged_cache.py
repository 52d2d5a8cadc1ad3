"""The paged-cache operators' checks of their arguments (before any CUDA call),
and the plain forms that the GPU tests hold them to.  No GPU needed."""
import math

import pytest
import torch

import gqa_attention_kv_split_gb300 as gqa
import paged_reference as R
from gqa_attention_kv_split_gb300 import build_lib


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()


def fake(shape, dtype=torch.bfloat16, **kw):
    return torch.zeros(shape, dtype=dtype, **kw)


def append_args(T=3, hq=4, hkv=2, d=64, page=16, dtype=torch.bfloat16, cache=None, P=5, B=3, mp=2):
    return dict(q=fake((T, hq, d), dtype), k=fake((T, hkv, d), dtype), v=fake((T, hkv, d), dtype),
                k_pages=fake((P, hkv, page, d), cache or dtype), v_pages=fake((P, hkv, page, d), cache or dtype),
                block_table=fake((B, mp), torch.int32), kv_lens=fake((B,), torch.int32))


@pytest.mark.parametrize("change,match", [
    (dict(q=torch.zeros(3, 4, 64)), "q has dtype f32; expected bf16"),
    (dict(q=fake((3, 4, 64), torch.float16)), "q has dtype f16; expected bf16"),
    (dict(v=fake((3, 2, 32))), "v has extent 32 in dimension 2; expected 64"),
    (dict(k=fake((3, 2, 96)), v=fake((3, 2, 96))), "head dim 96 is not 64, 128 or 256"),
    (dict(k=fake((3, 2, 128))[..., ::2]), "k: the last dimension is not dense"),
    (dict(k=fake((3, 2, 68))[..., :64]), "k: stride 68 in dimension 1 is not a multiple of 16 bytes"),
    (dict(k_pages=fake((5, 2, 16, 64), torch.float16)), "k_pages has dtype f16; expected bf16 or e4m3 or u8"),
    (dict(v_pages=fake((5, 2, 16, 64), torch.float8_e4m3fn)), "v_pages has dtype e4m3; expected bf16"),
    (dict(v_pages=fake((5, 2, 32, 64))), "v_pages has extent 32 in dimension 2; expected 16"),
    (dict(k_pages=fake((1, 2, 16, 64)).expand(5, 2, 16, 64)), "k_pages overlaps itself"),
    (dict(k_pages=fake((5, 1, 16, 64))), "k_pages has extent 1 in dimension 1; expected 2"),
    (dict(kv_lens=fake((3,), torch.int64)), "kv_lens has dtype unknown"),
    (dict(kv_lens=fake((2,), torch.int32), block_table=fake((2, 2), torch.int32)), "without qo_indptr there is one token per sequence"),
    (dict(qo_indptr=fake((3,), torch.int32)), "qo_indptr has extent 3 in dimension 0; expected 4"),
    (dict(rope=torch.zeros(8, 24)), "rope has 24 columns; a multiple of 16"),
    (dict(rope=torch.zeros(8, 128)), "rope has 128 columns"),
    (dict(rope=torch.zeros(8, 64, dtype=torch.float64)), "rope has dtype unknown"),
    (dict(k_scale=2.0), "belong to E4M3 pages"),
    (dict(k_scale=0.0), "k_scale must be finite and > 0"),
    (dict(v_scale=math.nan), "v_scale must be finite and > 0"),
    (dict(q_out=fake((3, 4, 64), torch.float16)), "q_out has dtype f16"),
    (dict(q=None, q_out=fake((3, 4, 64))), "q and q_out go together"),
    (dict(), "gqa_paged_append takes device tensors only"),
])
def test_append_refusals(change, match):
    with pytest.raises(gqa.GqaError, match=match):
        gqa.gqa_paged_append(**{**append_args(), **change})


def test_append_in_place_needs_the_same_strides():
    a = append_args()
    wide = fake((3, 8, 64))
    with pytest.raises(gqa.GqaError, match="q_out may be q itself, with q's type and strides"):
        gqa.gqa_paged_append(**{**a, "q": wide[:, :4], "q_out": wide.view(-1)[:3 * 4 * 64].view(3, 4, 64)})


def test_nvfp4_append_in_place_is_refused():
    a = nvfp4_args()
    with pytest.raises(gqa.GqaError, match="q_out may be q itself, with q's type and strides"):
        gqa.nvfp4_paged_append(**{**a, "q_out": a["q"].view(torch.uint8)[..., :128]})


def test_append_of_nothing_is_accepted():
    a = append_args(T=0)
    out = gqa.gqa_paged_append(**a, qo_indptr=fake((4,), torch.int32))
    assert out.shape == (0, 4, 64)


def nvfp4_args(T=2, P=3, B=2):
    return dict(q=fake((T, 32, 128)), k=fake((T, 8, 128)), v=fake((T, 8, 128)), k_fp4=fake((P, 8, 64, 64), torch.uint8),
                k_sf=fake((P, 8, 64, 8), torch.uint8), v_fp4=fake((P, 8, 64, 64), torch.uint8),
                v_sf=fake((P, 8, 64, 8), torch.float8_e4m3fn), block_table=fake((B, 2), torch.int32),
                qo_indptr=fake((B + 1,), torch.int32), kv_lens=fake((B,), torch.int32))


@pytest.mark.parametrize("change,match", [
    (dict(q=fake((2, 16, 128))), "q has extent 16 in dimension 1; expected 32"),
    (dict(k=fake((2, 4, 128))), "k has extent 4 in dimension 1; expected 8"),
    (dict(k=fake((2, 8, 64))), "k has extent 64 in dimension 2; expected 128"),
    (dict(k_sf=fake((2, 8, 64, 8), torch.uint8)), "k_sf has extent 2 in dimension 0; expected 3"),
    (dict(v_fp4=fake((3, 8, 64, 64), torch.bfloat16)), "v_fp4 has dtype bf16; expected u8"),
    (dict(v_fp4=fake((3, 8, 64, 128), torch.uint8)[..., ::2]), "v_fp4 is not dense"),
    (dict(rope=torch.zeros(4, 48)), "a multiple of 32"),
    (dict(q_scale=-1.0), "q_scale must be finite and > 0"),
    (dict(q_out=fake((2, 32, 128))), "q_out has dtype bf16; expected e4m3 or u8"),
    (dict(), "nvfp4_paged_append takes device tensors only"),
])
def test_nvfp4_append_refusals(change, match):
    with pytest.raises(gqa.GqaError, match=match):
        gqa.nvfp4_paged_append(**{**nvfp4_args(), **change})


def attn_args(B=2, hq=4, hkv=2, d=64, page=16, dtype=torch.float16, cache=None, P=5, mp=2):
    return dict(q=fake((B, hq, d), dtype), k_pages=fake((P, hkv, page, d), cache or dtype),
                v_pages=fake((P, hkv, page, d), cache or dtype), block_table=fake((B, mp), torch.int32),
                seq_lens=fake((B,), torch.int32), workspace=torch.zeros(16 << 20, dtype=torch.uint8))


@pytest.mark.parametrize("change,match", [
    (dict(q=torch.zeros(2, 4, 64)), "q has dtype f32; expected f16 or bf16"),
    (dict(q=fake((2, 4, 64))), "k_pages has dtype f16; expected bf16 or e4m3"),
    (dict(q=fake((2, 5, 64), torch.float16)), "5 query heads over 2 KV heads"),
    (dict(q=fake((2, 4, 32), torch.float16)), "k_pages has extent 64 in dimension 3; expected 32"),
    (dict(k_pages=fake((5, 2, 24, 64), torch.float16), v_pages=fake((5, 2, 24, 64), torch.float16)), "page size 24 is not"),
    (dict(v_pages=fake((5, 2, 16, 64), torch.uint8)), "v_pages has dtype u8; expected f16"),
    (dict(k_pages=fake((5, 2, 16, 128), torch.float16)[..., ::2]), "k_pages: the last dimension is not dense"),
    (dict(seq_lens=fake((3,), torch.int32)), "seq_lens has extent 3 in dimension 0; expected 2"),
    (dict(block_table=fake((2, 4), torch.int32)[:, ::2]), "block_table is not dense"),
    (dict(out=fake((2, 4, 64))), "out has dtype bf16; expected f16"),
    (dict(lse=torch.zeros(2, 2)), "lse has extent 2 in dimension 1; expected 4"),
    (dict(window=-1), "window -1 is negative"),
    (dict(softcap=-1.0), "softcap must be finite and >= 0"),
    (dict(q_scale=math.inf), "q_scale is not finite"),
    (dict(k_scale=math.inf), "k_scale must be finite and > 0"),
    (dict(k_scale=0.0), "k_scale must be finite and > 0"),
    (dict(workspace=torch.zeros(64, dtype=torch.uint8)), "workspace of 64 bytes"),
    (dict(), "gqa_paged_attn takes device tensors only"),
    (dict(workspace=None), "gqa_paged_attn takes device tensors only"),
])
def test_attention_refusals(change, match):
    with pytest.raises(gqa.GqaError, match=match):
        gqa.gqa_paged_attn(**{**attn_args(), **change})


def test_workspace_has_to_be_bytes():
    with pytest.raises(ValueError, match="dense 1-d uint8"):
        gqa.gqa_paged_attn(**{**attn_args(), "workspace": torch.zeros(1 << 20)})


def test_binding_takes_tensors_only():
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        gqa.gqa_paged_append(**{**append_args(), "q": [1.0], "q_out": fake((3, 4, 64))})
    with pytest.raises(ValueError, match="k has more than 6 dimensions"):
        gqa.gqa_paged_append(**{**append_args(), "k": fake((1,) * 7)})
    with pytest.raises(TypeError):
        gqa.gqa_paged_attn(**attn_args(), q_scale="1")
    with pytest.raises(OverflowError):
        gqa.gqa_paged_attn(**attn_args(), window=1 << 40)


def test_attention_refuses_other_head_dims():
    with pytest.raises(gqa.GqaError, match="head dim 96 is not 64, 128 or 256"):
        gqa.gqa_paged_attn(**attn_args(d=96))


def test_workspace_is_bounded_by_the_head_layout():
    n = gqa.gqa_paged_attn_workspace
    assert 0 < n(32, 8, 128) < n(64, 4, 128) < n(64, 4, 256) < 6 << 20
    assert n(5, 2, 128) == n(4, 0, 128) == n(8, 8, 96) == 0


# ---- the plain forms ---------------------------------------------------------

def test_reference_positions_and_rotation():
    assert R.positions(5, [4, 0, 1], [0, 3, 3, 4]) == [(0, 1), (0, 2), (0, 3), (2, 0), None]
    rope = torch.tensor([[0.0, 1.0]]).repeat(2, 1)  # a quarter turn of the first pair
    x = torch.arange(8, dtype=torch.float64).view(1, 1, 8)
    assert R.rotate(x[0], rope[0], False)[0, :4].tolist() == [-1.0, 0.0, 2.0, 3.0]


def test_reference_quantisation_ties_go_to_the_even_code():
    x = torch.zeros(16)
    x[0] = 6.0  # scale 1
    for i, (v, want) in enumerate([(0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0), (3.5, 4.0), (5.0, 4.0), (-0.75, -1.0)]):
        x[i + 1] = v
    val, sf = R.nvfp4_quantise(x)
    assert sf.item() == 1.0
    assert val[1:9].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -1.0]


def test_the_check_sees_a_planted_mistake():
    """A reference with one key too many is outside the bound that the GPU outputs are held to."""
    g = torch.Generator().manual_seed(1)
    q = torch.randn(1, 2, 64, generator=g).half()
    k, v = torch.randn(3, 1, 16, 64, generator=g).half(), torch.randn(3, 1, 16, 64, generator=g).half()
    table, lens = torch.tensor([[2, 0, 1]], dtype=torch.int32), torch.tensor([40], dtype=torch.int32)
    out, lse, _, _ = R.attention(q, k, v, table, lens)
    R.check_attention(out.half(), lse.float(), q, k, v, table, lens)
    with pytest.raises(AssertionError):
        R.check_attention(out.half(), lse.float(), q, k, v, table, lens + 1)
