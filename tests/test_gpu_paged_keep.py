"""GPU: gqa_paged_keep against rows moved one by one."""
import random

import pytest
import torch

import gqa_attention_kv_split_gb300 as gqa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def tensors(num, page, heads, widths, layers=0, nhd=False, seed=0):
    """Page tensors (dtype, width) with distinct bytes, head- or token-major."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for dtype, w in widths:
        esz = torch.empty(0, dtype=dtype).element_size()
        shape = (num, page, heads, w * esz) if nhd else (num, heads, page, w * esz)
        raw = torch.randint(0, 256, ((layers,) if layers else ()) + shape, generator=g, dtype=torch.uint8)
        t = raw.to(DEV).view(dtype)
        out.append(t.transpose(-3, -2) if nhd else t)
    return out


def as_bytes(t):
    """[..., heads, page, bytes] on the CPU."""
    nhd = t.stride(-2) > t.stride(-3)
    x = (t.transpose(-3, -2) if nhd else t).contiguous().view(torch.uint8).cpu()
    return x.transpose(-3, -2) if nhd else x


def moved(t, table, lens, indptr, kept, counts, page):
    """The plain form, on bytes."""
    x = as_bytes(t).clone()
    old = x.clone()
    for b, n in enumerate(counts):
        base = lens[b] - (indptr[b + 1] - indptr[b])
        for i in range(n):
            s, d = base + kept[b][i], base + i
            x[..., table[b][d // page], :, d % page, :] = old[..., table[b][s // page], :, s % page, :]
    return x


def check(drafts, cached, counts, page=16, heads=2, widths=((torch.bfloat16, 64),) * 2, layers=0, nhd=False, seed=0, extra=0):
    rng = random.Random(seed)
    B = len(drafts)
    lens, indptr = [n + c for n, c in zip(drafts, cached)], [0]
    for n in drafts:
        indptr.append(indptr[-1] + n)
    mp = max(1, max((n + page - 1) // page for n in lens)) + 1
    ids = list(range(B * mp))
    rng.shuffle(ids)
    table = [[ids[b * mp + p] if p * page < lens[b] else -5 for p in range(mp)] for b in range(B)]
    most = max(counts + [1]) + extra
    kept = [sorted(rng.sample(range(n), m)) + [-9] * (most - m) for n, m in zip(drafts, counts)]
    pages = tensors(B * mp, page, heads, widths, layers, nhd, seed)
    want = [moved(t, table, lens, indptr, kept, counts, page) for t in pages]
    new = gqa.gqa_paged_keep(pages, i32(table), i32(indptr), i32(lens), i32(kept), i32(counts))
    assert new.tolist() == [c + m for c, m in zip(cached, counts)]
    for t, w in zip(pages, want):
        assert torch.equal(as_bytes(t), w)


@pytest.mark.parametrize("nhd", [False, True])
@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("layers", [0, 1, 3])
def test_rows_move_together(page, layers, nhd):
    check([16, 1, 0, 33, 7], [40, 0, 9, 100, 15], [5, 1, 0, 12, 7], page=page, layers=layers, nhd=nhd, seed=page + layers)


@pytest.mark.parametrize("widths", [((torch.float16, 128), (torch.float16, 128)), ((E4M3, 64), (E4M3, 64)),
                                    ((torch.uint8, 64), (torch.uint8, 8), (torch.uint8, 64), (E4M3, 8)),
                                    ((torch.bfloat16, 256),), ((torch.float32, 2), (torch.bfloat16, 12))])
@pytest.mark.parametrize("heads", [1, 8, 13])
def test_types_and_widths(widths, heads):
    check([20, 64], [50, 3], [6, 30], page=64, heads=heads, widths=widths, seed=heads)


def test_long_drafts_and_long_lists():
    """More kept tokens than are resolved at a time, dense and sparse, and columns that nothing needs."""
    check([1000, 600, 300], [7, 100, 0], [500, 600, 129], seed=1, extra=3)
    check([1000, 1000], [0, 33], [999, 256], page=16, nhd=True, layers=2, seed=2)


def test_many_sequences():
    rng = random.Random(3)
    drafts = [rng.randint(0, 20) for _ in range(700)]
    check(drafts, [rng.randint(0, 40) for _ in drafts], [rng.randint(0, n) for n in drafts], heads=1, seed=3)


def call(kept, counts, drafts, lens, table=None, page=16, indptr=None):
    B = len(lens)
    if indptr is None:
        indptr = [0]
        for n in drafts:
            indptr.append(indptr[-1] + n)
    pages = tensors(B * 2, page, 2, ((torch.bfloat16, 64),))
    before = as_bytes(pages[0]).clone()
    table = table or [[2 * b, 2 * b + 1] for b in range(B)]
    new = gqa.gqa_paged_keep(pages, i32(table), i32(indptr), i32(lens), i32(kept), i32(counts))
    word = gqa.gqa_check_device_errors(0)
    return new.tolist(), (as_bytes(pages[0]) != before).flatten(1).any(1).tolist(), word


@pytest.mark.parametrize("kept,count", [([3, 2], 2), ([2, 2], 2), ([-1, 2], 2), ([1, 6], 2), ([1, 2], 3), ([1, 2], -1)])
def test_lists_that_make_no_sense_leave_their_sequence(kept, count):
    new, changed, word = call([kept, [1, 2]], [count, 2], [6, 6], [20, 20])
    assert word == 2 and new == [20, 16]
    assert changed == [False, False, True, False] or changed == [False, False, True, True]


def test_more_kept_than_drafted():
    new, changed, word = call([[0, 1, 2]], [3], [2], [20])
    assert (new, word) == ([20], 2) and not any(changed)


def test_lengths_shorter_than_the_draft():
    new, changed, word = call([[1, 2]], [2], [6], [3])
    assert (new, word) == ([3], 2) and not any(changed)
    assert call([[1, 2]], [0], [6], [0]) == ([0], [False, False], 0)  # an inactive sequence of a padded batch


def test_offsets_that_fall():
    new, changed, word = call([[1, 2], [1, 2]], [2, 0], None, [20, 20], indptr=[0, 6, 3])
    assert word == 4 and new == [16, 20]


@pytest.mark.parametrize("table", [[[0, -1]], [[0, 99]]])
def test_pages_out_of_range_are_flagged(table):
    """Tokens 14 .. 19 are drafted; 15, 17 and 19 are kept: one within page 0, two from the page that is none."""
    new, changed, word = call([[1, 3, 5]], [3], [6], [20], table=table)
    assert word == 2 and new == [17] and changed == [True, False]


def test_positions_behind_the_table_are_flagged():
    new, changed, word = call([[1, 3, 30]], [3], [31], [40])
    assert word == 2 and changed == [True, False]


def test_captured_on_another_stream():
    pages = tensors(2, 16, 2, ((torch.bfloat16, 64),))
    table, indptr, lens, kept, count = i32([[0, 1]]), i32([0, 6]), i32([20]), i32([[1, 3]]), i32([2])
    new = torch.zeros(1, dtype=torch.int32, device=DEV)
    before = as_bytes(pages[0]).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gqa.gqa_paged_keep(pages, table, indptr, lens, kept, count, new_lens=new)
    graph.replay()
    torch.cuda.synchronize()
    assert new.tolist() == [16]
    assert torch.equal(as_bytes(pages[0]), moved_bytes(before))


def moved_bytes(x):
    """Tokens 14 .. 19 drafted, 15 and 17 kept: to 14 and 15."""
    y = x.clone()
    y[0, :, 14], y[0, :, 15] = x[0, :, 15], x[1, :, 1]
    return y
