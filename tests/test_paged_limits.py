"""The sizes that the paged-cache entry points refuse are the ones that include/gqa.h names."""
import os
import re

import pytest
import torch

import gqa_attention_kv_split_gb300 as gqa
from gqa_attention_kv_split_gb300 import build_lib
from test_paged_cache import append_args, fake, nvfp4_args

MOST = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()


def comment_of(entry):
    src = open(os.path.join(build_lib.INCLUDE, "gqa.h")).read()
    comments = [c for c in re.findall(r"/\*.*?\*/", src, flags=re.S) if re.match(r"/\*\s*\* " + entry + r" --", c)]
    assert len(comments) == 1
    return " ".join(re.sub(r"\n \*", " ", comments[0]).split())


def test_append_names_its_limits():
    text = comment_of("gqa_paged_append_t")
    assert "page_size 1 .. 2^20" in text and "batch 1 .. 2^20" in text


@pytest.mark.parametrize("page,match", [(MOST, "takes device tensors only"), (MOST + 1, "page size 1048577 outside")])
def test_append_page_sizes(page, match):
    pages = [torch.empty(1, 1, page, 64, dtype=torch.bfloat16) for _ in range(2)]
    with pytest.raises(gqa.GqaError, match=match):
        gqa.gqa_paged_append(**{**append_args(hq=1, hkv=1), "k_pages": pages[0], "v_pages": pages[1]})


@pytest.mark.parametrize("batch,match", [(MOST, "takes device tensors only"), (MOST + 1, "batch 1048577 outside"), (0, "kv_lens is a null pointer")])
def test_append_batches(batch, match):
    many = dict(block_table=fake((batch, 1), torch.int32), kv_lens=fake((batch,), torch.int32), qo_indptr=fake((batch + 1,), torch.int32))
    with pytest.raises(gqa.GqaError, match=match):
        gqa.gqa_paged_append(**{**append_args(), **many})
    with pytest.raises(gqa.GqaError, match=match):
        gqa.nvfp4_paged_append(**{**nvfp4_args(), **many})
