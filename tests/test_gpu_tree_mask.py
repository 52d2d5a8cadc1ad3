"""GPU: gqa_tree_mask against the walk up each token's tree."""
import random

import pytest
import torch

import draft_reference as DR
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


def forest(sizes, seed, shape="random"):
    rng, parents = random.Random(seed), []
    for n in sizes:
        parents += [rng.randint(-1, i - 1) if shape == "random" else i - 1 if shape == "chain" else -1 for i in range(n)]
    indptr = [0]
    for n in sizes:
        indptr.append(indptr[-1] + n)
    return parents, indptr


def check(sizes, lens, seed=0, shape="random", words=None, pad=0, **kw):
    parents, indptr = forest(sizes, seed, shape)
    words = words or (max(sizes + [1]) + 31) // 32
    total = len(parents) + pad
    mask = torch.full((total, words), 77, dtype=torch.int32, device=DEV)
    positions = torch.full((total,), 78, dtype=torch.int32, device=DEV)
    gqa.gqa_tree_mask(i32(parents + [0] * pad), i32(indptr), i32(lens), mask=mask, positions=positions, **kw)
    want = DR.trees(parents, indptr, lens, **kw)
    n = len(parents)
    assert positions[:n].tolist() == [p for p, _ in want]
    assert mask[:n].tolist() == [DR.words_of(s, words) for _, s in want]
    assert (mask[n:] == 77).all() and (positions[n:] == 78).all()  # rows behind the last sequence


@pytest.mark.parametrize("shape", ["random", "chain", "flat"])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 200, 1024])
def test_sizes(n, shape):
    check([n], [n + 10], seed=n, shape=shape)


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 0), (3, 4), (5, 1000), (64, 0), (0, 7)])
@pytest.mark.parametrize("shape", ["random", "chain"])
def test_windows(window, sinks, shape):
    check([40, 1, 0, 17], [42, 1, 5, 517], seed=window, shape=shape, window=window, sinks=sinks)


def test_batches_padding_and_wide_masks():
    rng = random.Random(5)
    sizes = [rng.randint(0, 70) for _ in range(500)]
    check(sizes, [n + rng.randint(0, 3000) for n in sizes], seed=1, words=3, pad=9)
    check([5], [5], words=32)


def test_sequences_shorter_than_their_draft():
    """Positions are counted from where the draft would begin."""
    check([4, 3], [0, 1], seed=2)


def test_default_outputs():
    mask, positions = gqa.gqa_tree_mask(i32([-1, 0, 0, 1]), i32([0, 4]), i32([9]), max_tokens=4)
    assert mask.tolist() == [[1], [3], [5], [11]] and positions.tolist() == [5, 6, 6, 7]


def run(parents, indptr, lens, words=1):
    mask = torch.full((len(parents), words), 77, dtype=torch.int32, device=DEV)
    positions = torch.full((len(parents),), 78, dtype=torch.int32, device=DEV)
    gqa.gqa_tree_mask(i32(parents), i32(indptr), i32(lens), mask=mask, positions=positions)
    return mask, positions, gqa.gqa_check_device_errors(0)


def test_parents_out_of_range_count_as_none():
    mask, positions, word = run([-1, 1, 0, -2, 2 ** 31 - 1, 2], [0, 6], [6])
    assert word == 2
    assert mask[:, 0].tolist() == [1, 2, 5, 8, 16, 37] and positions.tolist() == [0, 0, 1, 0, 0, 2]


def test_trees_larger_than_the_mask():
    mask, positions, word = run([-1] + list(range(33)), [0, 34], [40])
    assert word == 2
    assert positions[:32].tolist() == list(range(6, 38)) and (positions[32:] == 78).all() and (mask[32:] == 77).all()


@pytest.mark.parametrize("indptr", [[0, 5, 3], [-1, 2, 5], [2, 4, 5], [0, 4, 9]])
def test_offsets_are_looked_at(indptr):
    mask, positions, word = run([-1] * 5, indptr, [9, 9])
    assert word == 4


def test_captured_and_replayed():
    parents, indptr, lens = i32([-1, 0, -1]), i32([0, 2, 3]), i32([5, 9])
    mask, positions = torch.zeros(3, 1, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gqa.gqa_tree_mask(parents, indptr, lens, mask=mask, positions=positions)
    lens.copy_(i32([7, 3]))
    parents.copy_(i32([-1, -1, -1]))
    graph.replay()
    torch.cuda.synchronize()
    assert mask[:, 0].tolist() == [1, 2, 1] and positions.tolist() == [5, 5, 2]
