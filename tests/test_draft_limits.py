"""The limits on a call's work that keep a block's share of it within 31 bits, from both sides: descriptors of tensors
that no machine holds, which are looked at before any memory is.  No GPU needed."""
import ctypes

import pytest

import gqa_attention_kv_split_gb300 as gqa
from gqa_attention_kv_split_gb300 import build_lib

F16, I32 = 1, 4
TOO_MANY, HOST = "too many", "device tensors only"


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()


def desc(dtype, *shape):
    """A dense host tensor of which only the descriptor is there."""
    d = gqa.GqaTensor()
    d.data, d.dtype, d.device, d.ndim = 1 << 20, dtype, -1, len(shape)
    stride = 1
    for i in reversed(range(len(shape))):
        d.shape[i], d.strides[i] = shape[i], stride
        stride *= shape[i]
    return d


def refusal(call, *args):
    L = gqa.lib()
    L.gqa_last_error.restype = ctypes.c_char_p
    st = call(*[ctypes.byref(a) if isinstance(a, gqa.GqaTensor) else a for a in args])
    assert st != 0
    return L.gqa_last_error().decode()


def tree(batch, total, hq, hkv, max_pages, page=256, d=64):
    pages = [desc(F16, 5, hkv, page, d) for _ in range(2)]
    return refusal(gqa.lib().gqa_paged_tree_attn_t, desc(F16, total, hq, d), *pages, desc(I32, batch, max_pages),
                   desc(I32, batch + 1), desc(I32, batch), None, None, desc(F16, total, hq, d), None, 1.0, 1.0, 1.0, 0, 0, 0.0,
                   None, 0, None)


# KV heads x (sequences + tokens x group / 128) x (capacity / 64 + 16) is 2^38 at most
@pytest.mark.parametrize("hkv,hq,batch,total,max_pages,match", [
    (8, 8, 32767, 128, 262140, HOST),  # 8 x 32768 x 2^20
    (8, 8, 32768, 128, 262140, TOO_MANY),
    (8, 8, 32767, 256, 262140, TOO_MANY),
    (8, 8, 32767, 128, 262141, TOO_MANY),
    (1, 1, 65535, 128, 1048572, HOST),  # 65536 x 2^22
    (1, 1, 65535, 256, 1048572, TOO_MANY),
    (1, 64, 1, 262142, 524284, HOST),  # tokens rather than sequences: 2^17 x 2^21
    (1, 64, 2, 262142, 524284, TOO_MANY),
    (1, 1024, 1, (1 << 21) - 1, 1, HOST),  # rows of a KV head: less than 2^31
    (1, 1024, 1, 1 << 21, 1, TOO_MANY),
])
def test_work_of_a_tree_attention(hkv, hq, batch, total, max_pages, match):
    assert match in tree(batch, total, hq, hkv, max_pages)


# sequences x KV heads x blocks of 8 heads x (capacity / 32 + 16) is 2^38 at most
@pytest.mark.parametrize("hkv,hq,batch,max_pages,match", [
    (8, 32, 32768, 131070, HOST),  # 2^18 x 2^20
    (8, 32, 32769, 131070, TOO_MANY),
    (8, 32, 32768, 131071, TOO_MANY),
    (1, 16, 65535, 262142, HOST),  # two blocks of heads: 131070 x 2^21
    (1, 17, 65535, 262142, TOO_MANY),
])
def test_work_of_an_attention_with_sinks(hkv, hq, batch, max_pages, match):
    pages = [desc(F16, 5, hkv, 256, 64) for _ in range(2)]
    assert match in refusal(gqa.lib().gqa_paged_window_attn_t, desc(F16, batch, hq, 64), *pages, desc(I32, batch, max_pages),
                            desc(I32, batch), desc(F16, batch, hq, 64), None, 1.0, 1.0, 1.0, 64, 4, 0.0, None, 0, None)
