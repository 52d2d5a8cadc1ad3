"""What the operators of drafted tokens write may not lie where other blocks of the same call still read: such calls
are refused before any CUDA call.  No GPU needed."""
import pytest
import torch

import gqa_attention_kv_split_gb300 as gqa
from gqa_attention_kv_split_gb300 import build_lib
from test_draft_refusals import keep_args, mask_args
from test_paged_cache import fake

I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()


@pytest.mark.parametrize("name", ["num_kept", "kept", "block_table", "qo_indptr", "kv_lens"])
def test_new_lengths_over_other_inputs(name):
    """A sequence's first block writes its new length while the others read how many tokens are kept, and which."""
    a, memory = keep_args(), fake((16,), I32)
    mine = memory.as_strided(a[name].shape, a[name].stride(), 2)
    for start in (1, 2, 1 + mine.numel()):  # its first number, its first two, its last
        with pytest.raises(gqa.GqaError, match=f"new_lens (overlaps {name}|may not be kv_lens)"):
            gqa.gqa_paged_keep(**{**a, name: mine}, new_lens=memory[start:start + 2])


def test_new_lengths_beside_other_inputs():
    """Neighbours in one allocation are no overlap."""
    memory = fake((8,), I32)
    a = {**keep_args(), "num_kept": memory[2:4]}
    for new_lens in (memory[0:2], memory[4:6]):
        with pytest.raises(gqa.GqaError, match="device tensors only"):
            gqa.gqa_paged_keep(**a, new_lens=new_lens)


@pytest.mark.parametrize("written", ["mask", "positions"])
@pytest.mark.parametrize("name", ["parents", "qo_indptr", "kv_lens", "mask"])
def test_masks_and_positions_over_other_arguments(name, written):
    """A tree's block writes its rows while the blocks of other trees read their parents, offsets and lengths."""
    if name == written:
        return
    a, memory = mask_args(), fake((16,), I32)
    other = memory.as_strided(a[name].shape, a[name].stride(), 6)
    for start in (2, 5 + other.numel()):  # its first number is in it, its last one
        out = memory.as_strided(a[written].shape, a[written].stride(), start)
        with pytest.raises(gqa.GqaError, match="mask overlaps positions" if name == "mask" else f"{written} overlaps {name}"):
            gqa.gqa_tree_mask(**{**a, name: other, written: out})


def test_positions_in_place_of_parents():
    """A tree's parents have been read when its positions are written: they may be the same tensor."""
    a = mask_args()
    with pytest.raises(gqa.GqaError, match="device tensors only"):
        gqa.gqa_tree_mask(**{**a, "positions": a["parents"]})
