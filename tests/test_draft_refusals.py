"""The checks that the operators of drafted tokens make of their arguments (before any CUDA call).  No GPU needed."""
import math

import pytest
import torch

import draft_reference as DR
import gqa_attention_kv_split_gb300 as gqa
from gqa_attention_kv_split_gb300 import build_lib
from test_paged_cache import append_args, attn_args, fake, nvfp4_args

I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()


@pytest.mark.parametrize("change,match", [
    (dict(q_norm=fake((32,))), "q_norm has extent 32 in dimension 0; expected 64"),
    (dict(q_norm=fake((64,), torch.float16)), "q_norm has dtype f16; expected bf16 or f32"),
    (dict(q_norm=fake((64,)), k_norm=torch.zeros(64)), "k_norm has dtype f32; expected bf16"),
    (dict(k_norm=fake((128,))[::2]), "k_norm is not dense"),
    (dict(q=None, q_norm=fake((64,))), "q_norm without q"),
    (dict(q_norm=fake((64,)), norm_eps=-1e-6), "norm_eps must be finite and >= 0"),
    (dict(k_norm=fake((64,)), norm_eps=math.nan), "norm_eps must be finite and >= 0"),
    (dict(positions=fake((3,), I32)), "positions are rows of the rope table: there is none"),
    (dict(positions=fake((2,), I32), rope=torch.zeros(8, 64)), "positions has extent 2 in dimension 0; expected 3"),
    (dict(positions=fake((3,), torch.int64), rope=torch.zeros(8, 64)), "positions has dtype unknown"),
    (dict(q_norm=fake((64,))), "gqa_paged_append takes device tensors only"),
])
def test_norm_append_refusals(change, match):
    with pytest.raises(gqa.GqaError, match=match):
        gqa.gqa_paged_append(**{**append_args(), **change})


@pytest.mark.parametrize("change,match", [
    (dict(k_norm=fake((64,))), "k_norm has extent 64 in dimension 0; expected 128"),
    (dict(positions=fake((2,), I32)), "positions are rows of the rope table"),
    (dict(q_norm=torch.zeros(128)), "nvfp4_paged_append takes device tensors only"),
])
def test_nvfp4_norm_append_refusals(change, match):
    with pytest.raises(gqa.GqaError, match=match):
        gqa.nvfp4_paged_append(**{**nvfp4_args(), **change})


def test_norm_append_of_nothing_is_accepted():
    a = append_args(T=0)
    out = gqa.gqa_paged_append(**a, qo_indptr=fake((4,), I32), rope=torch.zeros(8, 64), positions=fake((0,), I32), q_norm=fake((64,)))
    assert out.shape == (0, 4, 64)


def test_sinks_refusals():
    with pytest.raises(gqa.GqaError, match="sinks -1 is negative"):
        gqa.gqa_paged_attn(**attn_args(), window=4, sinks=-1)
    with pytest.raises(OverflowError):
        gqa.gqa_paged_attn(**attn_args(), window=4, sinks=1 << 40)
    with pytest.raises(gqa.GqaError, match="device tensors only"):
        gqa.gqa_paged_attn(**attn_args(), window=4, sinks=4)


def mask_args(T=5, B=2, words=1):
    return dict(parents=fake((T,), I32), qo_indptr=fake((B + 1,), I32), kv_lens=fake((B,), I32), mask=fake((T, words), I32),
                positions=fake((T,), I32))


@pytest.mark.parametrize("change,match", [
    (dict(parents=fake((5,), torch.int64)), "parents has dtype unknown"),
    (dict(qo_indptr=fake((2,), I32)), "qo_indptr has extent 2 in dimension 0; expected 3"),
    (dict(kv_lens=fake((0,), I32), qo_indptr=fake((1,), I32)), "kv_lens is a null pointer|batch 0"),
    (dict(mask=fake((4, 1), I32)), "mask has extent 4 in dimension 0; expected 5"),
    (dict(mask=fake((5, 33), I32)), "33 words of bits: 1 to 32"),
    (dict(mask=fake((5, 2), I32)[:, ::2]), "mask is not dense"),
    (dict(positions=fake((6,), I32)), "positions has extent 6"),
    (dict(window=-1), "window -1 is negative"),
    (dict(sinks=-2), "sinks -2 is negative"),
    (dict(), "gqa_tree_mask takes device tensors only"),
])
def test_tree_mask_refusals(change, match):
    with pytest.raises(gqa.GqaError, match=match):
        gqa.gqa_tree_mask(**{**mask_args(), **change})


def test_tree_mask_needs_a_size():
    a = mask_args()
    with pytest.raises(ValueError, match="max_tokens"):
        gqa.gqa_tree_mask(a["parents"], a["qo_indptr"], a["kv_lens"])
    with pytest.raises(gqa.GqaError, match="0 words|mask"):
        gqa.gqa_tree_mask(a["parents"], a["qo_indptr"], a["kv_lens"], max_tokens=0)


def test_tree_mask_of_nothing_is_accepted():
    mask, positions = gqa.gqa_tree_mask(fake((0,), I32), fake((3,), I32), fake((2,), I32), max_tokens=40)
    assert mask.shape == (0, 2) and positions.shape == (0,)


def tree_args(B=2, T=5, hq=4, hkv=2, d=64, page=16, dtype=torch.float16, cache=None, P=5, mp=2):
    return dict(q=fake((T, hq, d), dtype), k_pages=fake((P, hkv, page, d), cache or dtype), v_pages=fake((P, hkv, page, d), cache or dtype),
                block_table=fake((B, mp), I32), qo_indptr=fake((B + 1,), I32), kv_lens=fake((B,), I32), mask=fake((T, 1), I32),
                workspace=torch.zeros(64 << 20, dtype=torch.uint8))


@pytest.mark.parametrize("change,match", [
    (dict(q=torch.zeros(5, 4, 64)), "q has dtype f32; expected f16 or bf16"),
    (dict(q=fake((5, 5, 64), torch.float16)), "5 query heads over 2 KV heads"),
    (dict(q=fake((5, 4, 32), torch.float16)), "k_pages has extent 64 in dimension 3; expected 32"),
    (dict(q=fake((5, 4, 68), torch.float16)[..., :64]), "q: stride 68 in dimension 1"),
    (dict(k_pages=fake((5, 2, 24, 64), torch.float16), v_pages=fake((5, 2, 24, 64), torch.float16)), "page size 24 is not"),
    (dict(v_pages=fake((5, 2, 16, 64), torch.uint8)), "v_pages has dtype u8; expected f16"),
    (dict(qo_indptr=fake((2,), I32)), "qo_indptr has extent 2 in dimension 0; expected 3"),
    (dict(block_table=fake((3, 2), I32)), "block_table has extent 3 in dimension 0; expected 2"),
    (dict(mask=fake((4, 1), I32)), "mask has extent 4 in dimension 0; expected 5"),
    (dict(mask=fake((5, 33), I32)), "33 words of bits"),
    (dict(mask=fake((5, 1), torch.uint8)), "mask has dtype u8; expected i32"),
    (dict(window=4), "a window over a tree needs the tokens' positions"),
    (dict(positions=fake((4,), I32)), "positions has extent 4"),
    (dict(out=fake((5, 4, 64))), "out has dtype bf16; expected f16"),
    (dict(lse=torch.zeros(5, 2)), "lse has extent 2 in dimension 1; expected 4"),
    (dict(mask=None, window=-1), "window -1 is negative"),
    (dict(sinks=-1), "sinks -1 is negative"),
    (dict(softcap=math.nan), "softcap must be finite and >= 0"),
    (dict(q_scale=math.inf), "q_scale is not finite"),
    (dict(v_scale=0.0), "v_scale must be finite and > 0"),
    (dict(workspace=torch.zeros(64, dtype=torch.uint8)), "workspace of 64 bytes"),
    (dict(), "gqa_paged_tree_attn takes device tensors only"),
    (dict(workspace=None, mask=None), "gqa_paged_tree_attn takes device tensors only"),
])
def test_tree_attention_refusals(change, match):
    with pytest.raises(gqa.GqaError, match=match):
        gqa.gqa_paged_tree_attn(**{**tree_args(), **change})


def test_tree_attention_over_too_much_is_refused():
    """Its blocks count the work of their shares in 31 bits."""
    a = tree_args(B=60000, mp=1, page=256)
    a["block_table"] = torch.zeros(1, dtype=I32).expand(60000 * 70000).as_strided((60000, 70000), (0, 0))
    with pytest.raises(gqa.GqaError, match="not dense"):
        gqa.gqa_paged_tree_attn(**a)


def test_tree_attention_workspace():
    need = gqa.gqa_paged_tree_attn_workspace(32, 8, 128)
    assert 152 * 2 * 128 * 520 <= need <= 152 * 2 * 128 * 520 + 65536
    assert gqa.gqa_paged_tree_attn_workspace(32, 5, 128) == 0 and gqa.gqa_paged_tree_attn_workspace(32, 8, 96) == 0


def keep_args(B=2, P=5, h=2, page=16, d=64, dtype=torch.bfloat16):
    return dict(pages=(fake((P, h, page, d), dtype), fake((P, h, page, d), dtype)), block_table=fake((B, 2), I32),
                qo_indptr=fake((B + 1,), I32), kv_lens=fake((B,), I32), kept=fake((B, 3), I32), num_kept=fake((B,), I32))


LENS = fake((2,), I32)


@pytest.mark.parametrize("change,match", [
    (dict(pages=()), "0 tensors of pages: 1 to 4"),
    (dict(pages=(fake((5, 16, 64)),)), r"pages\[0\] has 3 dimensions; expected 4 or 5"),
    (dict(pages=(fake((5, 2, 16, 64)), fake((4, 2, 16, 64)))), r"pages\[1\] has 4 pages of 16 tokens"),
    (dict(pages=(fake((5, 2, 16, 64)), fake((5, 2, 32, 64)))), r"pages\[1\] has 5 pages of 32 tokens"),
    (dict(pages=(fake((5, 2, 16, 6)),)), "rows of 12 bytes are no multiple of 8|stride 6 in dimension 2"),
    (dict(pages=(fake((1, 2, 16, 64)).expand(5, 2, 16, 64),)), r"pages\[0\] overlaps itself"),
    (dict(pages=(fake((5, 2, 16, 128))[..., ::2],)), "the last dimension is not dense"),
    (dict(pages=(fake((5, 2, 16, 64), torch.int64),)), r"pages\[0\] has dtype unknown"),
    (dict(pages=(fake((5, 0, 16, 64)),)), r"pages\[0\] is empty"),
    (dict(kept=fake((3, 3), I32)), "kept has extent 3 in dimension 0; expected 2"),
    (dict(num_kept=fake((2,), torch.int64)), "num_kept has dtype unknown"),
    (dict(kv_lens=LENS, new_lens=LENS), "new_lens may not be kv_lens"),
    (dict(), "gqa_paged_keep takes device tensors only"),
])
def test_keep_refusals(change, match):
    with pytest.raises(gqa.GqaError, match=match):
        gqa.gqa_paged_keep(**{**keep_args(), **change})


def test_keep_takes_a_tensor_once():
    p = fake((5, 2, 16, 64))
    with pytest.raises(gqa.GqaError, match=r"pages\[1\] is pages\[0\] again"):
        gqa.gqa_paged_keep(**{**keep_args(), "pages": (p, p)})


def test_keep_takes_up_to_four_tensors():
    with pytest.raises(TypeError, match="up to 4 tensors"):
        gqa.gqa_paged_keep(**{**keep_args(), "pages": tuple(fake((5, 2, 16, 64)) for _ in range(5))})


def test_plain_tree_by_hand():
    # 0 and 1 follow the cache, 2 and 3 follow 0, 4 follows 2
    t = DR.trees([-1, -1, 0, 0, 2], [0, 5], [12])
    assert t == [(7, {0}), (7, {1}), (8, {0, 2}), (8, {0, 3}), (9, {0, 2, 4})]
    assert DR.trees([-1, -1, 0, 0, 2], [0, 5], [12], window=2)[4] == (9, {2, 4})
    assert DR.trees([-1, -1, 0, 0, 2], [0, 5], [12], window=2, sinks=8)[4] == (9, {0, 2, 4})
    assert DR.words_of({0, 31, 33}, 2) == [1 - (1 << 31), 2]
    # the plain attention of one token under a window with sinks is that of the places listed
    assert DR.visible_one(10, 3, 2) == [0, 1, 7, 8, 9] and DR.visible_one(4, 3, 2) == [0, 1, 2, 3]
    assert DR.visible_rows([0, 2], [5], window=2, sinks=1) == [[0, 2, 3], [0, 3, 4]]
    assert DR.visible_rows([0, 2], [5], mask=[[1], [3]]) == [[0, 1, 2, 3], [0, 1, 2, 3, 4]]
