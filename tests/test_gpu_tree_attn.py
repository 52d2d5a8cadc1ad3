"""GPU: gqa_paged_tree_attn against the plain 64-bit form, within the bound that
draft_reference.check_attention derives."""
import random

import pytest
import torch

import draft_reference as DR
import gqa_attention_kv_split_gb300 as gqa
from test_gpu_sinks import clean, make
from test_gpu_tree_mask import forest, i32

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


class Batch:
    """Drafts over caches: inputs on the GPU, and what each row sees."""

    def __init__(self, drafts, lens, tree=True, window=0, sinks=0, pad=0, words=None, seed=0, shape="random", mask=None, **kw):
        self.window, self.sinks = window, sinks
        parents, self.indptr = forest(drafts, seed, shape)
        self.n = len(parents)
        self.mask = self.positions = None
        if tree:
            words = words or (max(drafts + [1]) + 31) // 32
            t = DR.trees(parents, self.indptr, lens, window, sinks)
            self.mask = mask or [DR.words_of(s, words) for _, s in t]
            self.positions = [p for p, _ in t]
        self.visible = DR.visible_rows(self.indptr, lens, window, sinks, self.mask, self.positions)
        seq = [b for b, n in enumerate(drafts) for _ in range(n)]
        # (every cached and drafted place is filled that some row of its sequence sees, or that is drafted: a token that
        # no mask shows is still there)
        filled = [sorted(set(v) | {t for t in range(max(0, lens[b] - drafts[b]), lens[b])}) for v, b in zip(self.visible, seq)]
        q, self.k, self.v, self.table, self.lens, _ = make(lens, filled, rows=seq, seed=seed, **kw)
        self.seq = seq
        if pad:
            q = torch.cat([q, torch.full((pad,) + q.shape[1:], float("nan"), dtype=q.dtype, device=DEV)])
            if tree:
                self.mask += [[-1] * len(self.mask[0])] * pad
                self.positions += [10 ** 9] * pad
        self.q = q

    def args(self):
        d = dict(q=self.q, k_pages=self.k, v_pages=self.v, block_table=self.table, qo_indptr=i32(self.indptr), kv_lens=self.lens,
                 window=self.window, sinks=self.sinks)
        if self.mask is not None:
            words = len(self.mask[0]) if self.mask else 1
            d.update(mask=i32(self.mask).view(-1, words), positions=i32(self.positions))
        return d

    def check(self, lse=True, **kw):
        T = self.q.shape[0]
        out = torch.full(self.q.shape, 5.0, dtype=self.q.dtype, device=DEV)
        l = torch.full((T, self.q.shape[1]), 9.0, device=DEV) if lse else None
        got = gqa.gqa_paged_tree_attn(**self.args(), out=out, lse=l, **kw)
        torch.cuda.synchronize()
        assert got is out
        assert (out[self.n:] == 5.0).all() and (l is None or (l[self.n:] == 9.0).all())  # rows behind the last sequence
        tables = self.table.cpu().clamp(min=0)[self.seq] if self.n else None
        DR.check_attention(out[:self.n], None if l is None else l[:self.n], self.q[:self.n], *clean(self.k, self.v), tables,
                           self.visible, **kw)
        return out, l


TYPES = [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)]


@pytest.mark.parametrize("d", [128, 64, 256])
@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("tree", [False, True])
def test_one_short_draft(tree, dtype, cache, d):
    Batch([3], [20], tree=tree, d=d, dtype=dtype, cache=cache, seed=d).check()


@pytest.mark.parametrize("d", [128, 64, 256])
@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("tree", [False, True])
def test_matches_plain_form(tree, dtype, cache, d):
    lens = [1, 2, 20, 64, 65, 127, 128, 129, 0, 200, 700, 300]
    drafts = [1, 2, 5, 16, 1, 33, 3, 8, 0, 70, 12, 40]
    Batch(drafts, lens, tree=tree, d=d, dtype=dtype, cache=cache, seed=d).check()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (4, 1), (7, 1), (8, 1), (16, 1), (17, 1), (40, 2), (32, 8), (12, 12)])
@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_groups_of_every_size(hq, hkv, cache):
    """Rows of a KV head below, at and above 32, 64 and 128: in four copies, two, one, and in several blocks."""
    Batch([3, 9, 17, 40, 0], [150, 33, 90, 300, 9], hq=hq, hkv=hkv, d=64, dtype=BF16, cache=cache, seed=hq).check()
    Batch([8], [190], hq=hq, hkv=hkv, d=128, dtype=BF16, cache=cache, seed=hq).check()
    Batch([31], [500], tree=False, hq=hq, hkv=hkv, d=128, dtype=BF16, cache=cache, seed=hq).check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, E4M3)])
def test_pages_and_layouts(page, layout, dtype, cache):
    for d in (64, 128, 256):
        Batch([5, 20, 1], [600, 33, 270], page=page, layout=layout, dtype=dtype, cache=cache, d=d, seed=page).check()


@pytest.mark.parametrize("window", [1, 5, 64, 129, 400, 5000])
@pytest.mark.parametrize("sinks", [0, 1, 16, 130, 9999])
@pytest.mark.parametrize("tree", [False, True])
def test_windows_and_sinks(window, sinks, tree):
    lens, drafts = [1, 17, 64, 200, 0, 900, 700], [1, 6, 20, 9, 0, 33, 5]
    Batch(drafts, lens, tree=tree, window=window, sinks=sinks, d=64, seed=window).check()
    Batch(drafts, lens, tree=tree, window=window, sinks=sinks, d=256, page=64, dtype=BF16, seed=sinks).check()
    Batch([20, 3], [700, 900], tree=tree, window=window, sinks=sinks, page=32, dtype=BF16, cache=E4M3, seed=sinks).check(k_scale=0.1, v_scale=0.2)


def test_scales_caps_and_signs():
    b = Batch([9, 30], [300, 40], d=128, dtype=BF16, seed=1, spread=3.0)
    b.check(q_scale=0.5, softcap=20.0)
    b.check(q_scale=-1.0)
    b.check(q_scale=-2.0, softcap=5.0)
    b.check(q_scale=0.0)
    b.check(lse=False, v_scale=3.0)
    Batch([9, 30], [300, 40], d=128, dtype=F16, cache=E4M3, seed=2).check(k_scale=0.06, v_scale=0.03, softcap=30.0)


def test_scales_next_to_nothing():
    """Rows of zeros and scales whose product with a row's own power of two would be 0: every token weighs the same."""
    for scale in (1e-30, 1e-38, 0.0):
        b = Batch([9, 3], [300, 40], d=64, dtype=BF16, cache=E4M3, seed=22)
        b.q[:5] = 0
        b.check(k_scale=1e-7, q_scale=scale)


def test_maxima_that_grow():
    """Keys whose scores rise along the sequence: the maximum in use is passed again and again, by a little and by a lot."""
    for dtype, cache in TYPES:
        for step in (0.02, 0.3):
            b = Batch([5, 40], [900, 700], d=128, dtype=dtype, cache=cache, seed=3)
            k = b.k.float()
            for i, n in enumerate([900, 700]):
                t = torch.arange(n, device=DEV)
                # (q . k grows with t for rows whose first element is positive, and falls for the others)
                at = b.table[i].long()[t // 16]
                k[at, :, t % 16, 0] = (t * step)[:, None].clamp(max=400.0)
            b.k.copy_(k.to(b.k.dtype))
            b.check()


def test_rows_that_see_nothing():
    # empty masks over an empty cache, and over one that has tokens
    Batch([3, 2], [3, 30], seed=4, mask=[[0], [2], [0], [0], [3]]).check()
    # drafts longer than what the cache holds: tokens without a place
    for tree in (False, True):
        Batch([5, 9], [3, 0], tree=tree, seed=5, shape="chain").check()
    out, lse = Batch([4], [0], seed=6).check()
    assert (out == 0).all() and (lse == float("-inf")).all()


def test_padding_and_wide_masks():
    Batch([3, 0, 7], [50, 9, 300], pad=5, words=4, seed=7).check()
    Batch([3, 0, 7], [50, 9, 300], tree=False, pad=5, seed=8).check()
    # bits of tokens that are not there
    b = Batch([3, 6], [20, 300], seed=9)
    b.mask = [[w | ~63 if b.seq[t] else w | ~7 for w in m] for t, m in enumerate(b.mask)]
    b.check()
    # a token behind the mask's words is seen by none, and sees none of its draft
    b = Batch([40], [100], shape="chain", words=1, seed=10)
    b.check()


def test_many_sequences():
    rng = random.Random(11)
    drafts = [rng.randint(0, 12) for _ in range(300)]
    Batch(drafts, [n + rng.randint(0, 60) for n in drafts], hq=8, hkv=4, d=64, dtype=BF16, seed=11).check()


@pytest.mark.parametrize("batch", [2, 31, 32, 33, 65])
def test_batches_of_every_size(batch):
    """Around the 32 sequences that a warp looks over at once: empty drafts, empty caches, short and split ones."""
    rng = random.Random(23 + batch)
    drafts = [rng.choice([0, 1, 5, 9]) for _ in range(batch)]
    lens = [rng.choice([0, n, n + 20, n + rng.randint(100, 900)]) for n in drafts]
    lens[batch // 2] = drafts[batch // 2] + 3000
    Batch(drafts, lens, hq=8, hkv=2, d=64, dtype=BF16, pad=2, seed=23).check()
    Batch(drafts, lens, tree=False, window=300, sinks=10, hq=6, hkv=3, d=64, dtype=F16, cache=E4M3, seed=24).check()


@pytest.mark.parametrize("batch", [5, 40])
def test_offsets_that_fall_leave_the_others(batch):
    b = Batch([3] * batch, [50 + i for i in range(batch)], hq=4, hkv=2, d=64, seed=25)
    want, _ = b.check()
    a = b.args()
    indptr = list(b.indptr)
    indptr[2] = b.n + 7  # the second sequence's end and the third one's start
    a["qo_indptr"] = i32(indptr)
    out = torch.full_like(b.q, 5.0)
    gqa.gqa_paged_tree_attn(**a, out=out)
    assert gqa.gqa_check_device_errors(0) == 4
    assert torch.equal(out[:3], want[:3]) and torch.equal(out[9:], want[9:]) and (out[3:9] == 5.0).all()


def test_capacities_up_to_the_limit():
    """Block tables for 2^30 tokens, of which a few pages are there."""
    b = Batch([6, 3], [700, 40], hq=16, hkv=8, d=64, page=256, seed=26)
    want, _ = b.check()
    a = b.args()
    wide = torch.full((2, 1 << 22), -1, dtype=torch.int32, device=DEV)
    wide[:, :b.table.shape[1]] = b.table
    a["block_table"] = wide
    got = gqa.gqa_paged_tree_attn(**a)
    # (the shares may be others: both are the same sums in another order)
    assert (got.double() - want.double()).abs().max() <= 2 * torch.finfo(F16).eps * max(1.0, want.double().abs().max().item())
    assert gqa.gqa_check_device_errors(0) == 0


@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, E4M3)])
def test_long_sequences_split_over_blocks(hkv, dtype, cache):
    Batch([6, 20, 3], [20000, 9000, 11], hq=4 * hkv, hkv=hkv, page=64, dtype=dtype, cache=cache, seed=12).check()
    Batch([50], [30000], hq=4 * hkv, hkv=hkv, page=64, dtype=dtype, cache=cache, d=64, seed=13).check()
    Batch([7], [25000], tree=False, window=9000, sinks=3000, hq=4 * hkv, hkv=hkv, page=32, dtype=dtype, cache=cache, d=256, seed=14).check()


def test_long_chains():
    """A chain of many row blocks, whose first ones see few of its tokens."""
    Batch([300, 5], [300, 40], tree=False, hq=8, hkv=2, d=64, dtype=BF16, seed=15).check()
    Batch([260], [1200], tree=False, hq=4, hkv=1, d=128, dtype=F16, seed=16).check()


def test_trees_of_many_words():
    Batch([1024], [1300], hq=2, hkv=1, d=64, dtype=F16, shape="chain", seed=27).check()
    Batch([200, 64], [200, 500], hq=4, hkv=2, d=64, dtype=BF16, seed=17).check()


def test_strided_queries_and_outputs():
    b = Batch([5, 9], [100, 30], hq=4, hkv=2, d=64, dtype=BF16, seed=18)
    wide = torch.zeros(14, 10, 64, dtype=BF16, device=DEV)
    wide[:, 3:7] = b.q
    want, _ = b.check()
    b.q = wide[:, 3:7]
    got = gqa.gqa_paged_tree_attn(**b.args())
    assert torch.equal(got, want)


def test_same_bits_every_time():
    b = Batch([20, 5, 64], [3000, 700, 9000], hq=8, hkv=2, d=128, dtype=BF16, seed=19)
    want = gqa.gqa_paged_tree_attn(**b.args())
    for _ in range(5):
        assert torch.equal(gqa.gqa_paged_tree_attn(**b.args()), want)


def test_bad_pages_and_offsets_are_flagged():
    b = Batch([4], [100], seed=20)
    a = b.args()
    a["block_table"] = a["block_table"].clone()
    a["block_table"][0, 2] = 10 ** 6
    gqa.gqa_paged_tree_attn(**a)
    assert gqa.gqa_check_device_errors(0) == 2
    for indptr, B in (([0, 5, 3], 2), ([-1, 2, 4], 2), ([2, 4, 4], 2), ([0, 4, 9], 2)):
        b = Batch([4], [100], seed=20)
        a = b.args()
        a.update(qo_indptr=i32(indptr), kv_lens=i32([100] * B), block_table=b.table.repeat(B, 1))
        out = torch.full_like(b.q, 5.0)
        gqa.gqa_paged_tree_attn(**a, out=out)
        assert gqa.gqa_check_device_errors(0) == 4, indptr


def test_nothing_to_do():
    b = Batch([0, 0], [10, 20], seed=21, hq=4)
    out = gqa.gqa_paged_tree_attn(**{**b.args(), "q": torch.zeros(0, 4, 128, dtype=F16, device=DEV), "mask": None, "positions": None})
    assert out.shape == (0, 4, 128)
