"""GPU: the operators of drafted tokens together, as a step with a draft makes them -- masks,
appends with norms at the tree's positions, attention of the tree, the accepted path kept -- over
many steps, captured into graphs, on other streams and from several threads."""
import ctypes
import random
import threading

import pytest
import torch

import draft_reference as DR
import gqa_attention_kv_split_gb300 as gqa
from test_gpu_paged_run import rope_table
from test_gpu_tree_attn import Batch
from test_gpu_tree_mask import forest, i32

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


class Model:
    """The attention of one layer of a model with normed heads: its cache, and what it appends for a token."""

    def __init__(self, B, hq=8, hkv=2, d=128, page=16, cap=512, dtype=BF16, cache=None, seed=0, window=0, sinks=0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.B, self.hq, self.hkv, self.d, self.page, self.dtype = g, B, hq, hkv, d, page, dtype
        self.cache, self.window, self.sinks = cache or dtype, window, sinks
        mp = cap // page
        self.table = torch.randperm(B * mp, generator=g).to(torch.int32).view(B, mp).to(DEV)
        self.rope = rope_table(cap, d).to(DEV)
        self.scales = (0.02, 0.01) if self.cache == E4M3 else (1.0, 1.0)
        self.norms = [(torch.rand(d, generator=g) + 0.5).to(dtype).to(DEV) for _ in range(2)]
        self.pages = self.new_pages()

    def new_pages(self):
        shape = (self.table.numel(), self.hkv, self.page, self.d)
        return [torch.full(shape, float("nan")).to(self.cache).to(DEV) for _ in range(2)]

    def rows(self, n):
        return torch.randn(n, self.hq + 2 * self.hkv, self.d, generator=self.g).to(self.dtype).to(DEV)

    def append(self, x, pages, lens, indptr, positions=None):
        q, k, v = x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]
        return gqa.gqa_paged_append(q, k, v, *pages, self.table, lens, qo_indptr=indptr, rope=self.rope, k_scale=self.scales[0],
                                    v_scale=self.scales[1], positions=positions, q_norm=self.norms[0], k_norm=self.norms[1])

    def kw(self):
        return dict(k_scale=self.scales[0], v_scale=self.scales[1], window=self.window, sinks=self.sinks)

    def tree(self, q, lens, indptr, mask, positions, **kw):
        return gqa.gqa_paged_tree_attn(q, *self.pages, self.table, indptr, lens, mask=mask, positions=positions, **self.kw(), **kw)

    def one(self, q, pages, lens, **kw):
        return gqa.gqa_paged_attn(q, *pages, self.table, lens, **self.kw(), **kw)

    def same_cache(self, other, lens):
        """The first lens[b] tokens of each sequence, byte for byte."""
        for p, o in zip(self.pages, other):
            p, o = (x.view(torch.uint8 if self.cache == E4M3 else torch.int16) for x in (p, o))
            for b, n in enumerate(lens):
                t = torch.arange(n, device=DEV)
                at = self.table[b].long()[t // self.page]
                if not torch.equal(p[at, :, t % self.page], o[at, :, t % self.page]):
                    return False
        return True


def path_to(parents, lo, j):
    path = []
    while j >= 0:
        path.append(j)
        j = parents[lo + j]
    return path[::-1]


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (BF16, E4M3)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_steps_with_drafts_are_steps_without(dtype, cache, window, sinks):
    """Decoding through trees of drafts, a random path of each accepted, leaves the cache that decoding token by token
    leaves, to the byte, and the accepted tokens' outputs are the one-token attention's: both are within half a step of the
    output's type and, by the weights' two terms and the scores, about 2^-16 + 2 * 2^-17 of the largest |v| of the exact
    value (paged_reference.check_attention), twice that apart; a score of up to 2^4 is off by 2^-19 of it."""
    rng = random.Random(1)
    m = Model(B=5, dtype=dtype, cache=cache, seed=3, window=window, sinks=sinks)
    plain = m.new_pages()
    lens = [30, 1, 64, 0, 100]
    x, indptr = m.rows(sum(lens)), i32([0, 30, 31, 95, 95, 195])
    m.append(x, m.pages, i32(lens), indptr)
    m.append(x, plain, i32(lens), indptr)
    for step in range(6):
        drafts = [rng.randint(1, 40) for _ in lens]
        parents, offsets = forest(drafts, 100 + step)
        full, indptr = [a + n for a, n in zip(lens, drafts)], i32(offsets)
        mask, positions = gqa.gqa_tree_mask(i32(parents), indptr, i32(full), max_tokens=40, window=window, sinks=sinks)
        x = m.rows(sum(drafts))
        q = m.append(x, m.pages, i32(full), indptr, positions)
        lse = torch.empty(sum(drafts), m.hq, device=DEV)
        out = m.tree(q, i32(full), indptr, mask, positions, lse=lse)
        # a path of each tree is accepted
        paths = [path_to(parents, offsets[b], rng.randrange(n)) if rng.random() < 0.8 else [] for b, n in enumerate(drafts)]
        kept = i32([p + [0] * (40 - len(p)) for p in paths])
        new = gqa.gqa_paged_keep(m.pages, m.table, indptr, i32(full), kept, i32([len(p) for p in paths]))
        # the same tokens one by one
        for k in range(max(len(p) for p in paths)):
            who = [b for b, p in enumerate(paths) if len(p) > k]
            rows = torch.tensor([offsets[b] + paths[b][k] for b in who], device=DEV)
            now = torch.tensor([lens[b] + k + 1 if b in who else 0 for b in range(5)])
            at = torch.zeros(5, dtype=torch.long, device=DEV)
            at[torch.tensor(who, device=DEV)] = rows
            q1 = m.append(x[at], plain, now.int().to(DEV), None)
            l1 = torch.empty(5, m.hq, device=DEV)
            o1 = m.one(q1, plain, now.int().to(DEV), lse=l1)
            assert torch.equal(q1[who], q[rows])
            mag = float(torch.nan_to_num(plain[1].float()).abs().max()) * m.scales[1]
            tol = torch.finfo(dtype).eps * o1[who].float().abs() + 2.0 ** -14 * mag
            assert ((out[rows].float() - o1[who].float()).abs() <= tol).all()
            assert ((lse[rows] - l1[who]).abs() <= 2.0 ** -16 * (1 + l1[who].abs())).all()
        lens = [a + len(p) for a, p in zip(lens, paths)]
        assert new.tolist() == lens
        assert m.same_cache(plain, lens)


def test_nvfp4_drafts_are_kept():
    """The codes and scales of accepted tokens, moved, are those of the tokens appended one after the other."""
    g = torch.Generator().manual_seed(5)
    n, base = 20, 50
    x = torch.randn(base + n, 48, 128, generator=g).bfloat16().to(DEV)
    parents, path = forest([n], 6)[0], None
    path = max((path_to(parents, 0, j) for j in range(n)), key=len)
    rope, w = rope_table(128, 128).to(DEV), torch.rand(128, generator=g).to(DEV)
    table = i32([[2, 0]])
    z = lambda k: torch.zeros(3, 8, 64, k, dtype=torch.uint8, device=DEV)

    def append(rows, cache, lens, positions=None):
        return gqa.nvfp4_paged_append(rows[:, :32], rows[:, 32:40], rows[:, 40:], *cache, table, i32([0, len(rows)]), i32([lens]), rope=rope,
                                      q_scale=0.02, positions=positions, q_norm=w, k_norm=w)
    drafted, plain = (z(64), z(8), z(64), z(8)), (z(64), z(8), z(64), z(8))
    for cache in (drafted, plain):
        append(x[:base], cache, base)
    mask, positions = gqa.gqa_tree_mask(i32(parents), i32([0, n]), i32([base + n]), max_tokens=n)
    append(x[base:], drafted, base + n, positions)
    new = gqa.gqa_paged_keep(drafted, table, i32([0, n]), i32([base + n]), i32([path]), i32([len(path)]))
    append(x[[base + j for j in path]], plain, base + len(path))
    assert new.tolist() == [base + len(path)]
    for a, b in zip(drafted, plain):
        for t in range(base + len(path)):
            assert torch.equal(a[int(table[0, t // 64]), :, t % 64], b[int(table[0, t // 64]), :, t % 64])


def test_captured_step():
    """One graph of a whole step, replayed with other trees, lengths and accepted paths."""
    m = Model(B=4, seed=7, cap=1024)
    lens = [300, 5, 64, 700]
    m.append(m.rows(sum(lens)), m.pages, i32(lens), i32([0, 300, 305, 369, 1069]))
    n = 12
    indptr = i32([0, 12, 24, 36, 48])
    parents, full, kept, count = i32([-1] * 48), i32([0] * 4), i32([[0] * n] * 4), i32([0] * 4)
    x = torch.zeros(48, m.hq + 2 * m.hkv, m.d, dtype=m.dtype, device=DEV)
    lse = torch.empty(48, m.hq, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mask, positions = gqa.gqa_tree_mask(parents, indptr, full, max_tokens=n)
        q = m.append(x, m.pages, full, indptr, positions)
        out = m.tree(q, full, indptr, mask, positions, lse=lse)
        new = gqa.gqa_paged_keep(m.pages, m.table, indptr, full, kept, count)
    rng = random.Random(2)
    for step in range(5):
        tree, offsets = forest([n] * 4, 50 + step)
        now = [a + n for a in lens]
        paths = [path_to(tree, offsets[b], rng.randrange(n)) for b in range(4)]
        for t, v in ((parents, tree), (full, now), (kept, [p + [0] * (n - len(p)) for p in paths]), (count, [len(p) for p in paths])):
            t.copy_(i32(v))
        x.copy_(m.rows(48))
        graph.replay()
        torch.cuda.synchronize()
        lens = [a + len(p) for a, p in zip(lens, paths)]
        assert new.tolist() == lens
        # the outputs against the cache as the attention saw it: the kept rows moved back to their drafted places
        pages = [p.clone() for p in m.pages]
        qs = m.append(x, pages, i32(now), indptr, positions)
        assert torch.equal(qs, q)
        clean = [torch.nan_to_num(p.float().cpu()).to(m.cache) for p in pages]
        bits = [s for _, s in DR.trees(tree, offsets, now)]
        visible = [list(range(now[t // n] - n)) + sorted(now[t // n] - n + j for j in bits[t]) for t in range(48)]
        DR.check_attention(out, lse, q, *clean, m.table.cpu()[[t // n for t in range(48)]], visible)


def batches():
    return [Batch([20, 3], [4000, 77], hq=16, hkv=1, page=64, dtype=BF16, seed=31),
            Batch([6, 40, 1], [9000, 300, 20], hq=8, hkv=2, page=64, dtype=BF16, seed=32),
            Batch([64], [6000], hq=32, hkv=8, page=64, dtype=BF16, cache=E4M3, seed=33),
            Batch([5, 5, 5, 5], [700, 30, 5000, 5], tree=False, hq=4, hkv=4, d=64, page=32, dtype=F16, seed=34)]


def test_two_graphs_replayed_at_once():
    bs = batches()[:2]
    want = [gqa.gqa_paged_tree_attn(**b.args()) for b in bs]
    graphs, outs, keep = [], [], []
    for b in bs:
        a = b.args()
        keep.append(a)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gqa.gqa_paged_tree_attn(**a))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(30):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_captured_call_without_workspace_is_refused_by_the_library():
    b = batches()[1]
    a = b.args()
    out = torch.empty_like(b.q)
    args = (a["q"], a["k_pages"], a["v_pages"], a["block_table"], a["qo_indptr"], a["kv_lens"], a["mask"], a["positions"], out, None,
            None, 1.0, 1.0, 1.0, 0, 0, 0.0)
    assert gqa._binding().tree_attn(*args) == 0
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a["kv_lens"].add_(0)  # (a graph with something in it)
        status = gqa._binding().tree_attn(*args)
    assert status == 7 and b"workspace of its own" in gqa.lib().gqa_last_error()
    gqa.gqa_release_workspace()
    again = gqa.gqa_paged_tree_attn(**a)
    torch.cuda.synchronize()
    assert torch.equal(again, out)


def in_threads(work, n):
    threads = [threading.Thread(target=work, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()


@pytest.mark.parametrize("shared", [False, True])
def test_threads_and_streams(shared):
    """Calls of several threads, on a stream each or all on one, give what one call gives."""
    bs = batches()
    args = [b.args() for b in bs]
    want = [gqa.gqa_paged_tree_attn(**a) for a in args]
    torch.cuda.synchronize()
    bad, start, one = [], threading.Barrier(4), torch.cuda.Stream()

    def work(i):
        stream = one if shared else torch.cuda.Stream()
        with torch.cuda.stream(stream):
            start.wait(60)
            outs = [gqa.gqa_paged_tree_attn(**args[i]).clone() for _ in range(40)]
        stream.synchronize()
        bad.extend(i for o in outs if not torch.equal(o, want[i]))
    in_threads(work, 4)
    assert not bad


def test_per_thread_streams_and_threads_that_end():
    """cudaStreamPerThread: one handle, a workspace for each thread, given back when the thread ends."""
    b = batches()[0]
    a, want = b.args(), gqa.gqa_paged_tree_attn(**b.args())
    outs = [torch.empty_like(want) for _ in range(4)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        d = [gqa._desc(t, "t") for t in (a["q"], a["k_pages"], a["v_pages"], a["block_table"], a["qo_indptr"], a["kv_lens"], a["mask"],
                                         a["positions"], outs[i])]
        st = gqa.lib().gqa_paged_tree_attn_t(*map(ctypes.byref, d), None, 1.0, 1.0, 1.0, 0, 0, 0.0, None, 0, ctypes.c_void_p(2))
        if st:
            bad.append(st)
    in_threads(work, 4)
    torch.cuda.synchronize()
    assert not bad and all(torch.equal(o, want) for o in outs)
    free = torch.cuda.mem_get_info(0)[0]
    for _ in range(10):
        in_threads(work, 1)
    torch.cuda.synchronize()
    assert free - torch.cuda.mem_get_info(0)[0] < 100 << 20  # (10 workspaces are 450 MB)


def test_own_workspace():
    b = batches()[1]
    need = gqa.gqa_paged_tree_attn_workspace(8, 2, 128)
    ws = torch.full((need + 256,), 0x7F, dtype=torch.uint8, device=DEV)  # (NaN wherever it is read before it is written)
    got = gqa.gqa_paged_tree_attn(**b.args(), workspace=ws[:need])
    assert torch.equal(got, gqa.gqa_paged_tree_attn(**b.args()))
    assert (ws[need:] == 0x7F).all()


def test_other_operators_between():
    """Attention right behind the append that fills its cache, and behind itself, with nothing waited for."""
    m = Model(B=3, seed=9, cap=512, cache=E4M3)
    lens = [400, 3, 77]
    m.append(m.rows(480), m.pages, i32(lens), i32([0, 400, 403, 480]))
    parents, offsets = forest([9, 20, 4], 3)
    full, indptr = i32([409, 23, 81]), i32(offsets)
    x = m.rows(33)
    mask, positions = gqa.gqa_tree_mask(i32(parents), indptr, full, max_tokens=20)
    q = m.append(x, m.pages, full, indptr, positions)
    torch.cuda.synchronize()
    want = m.tree(q, full, indptr, mask, positions)
    torch.cuda.synchronize()
    for _ in range(50):
        for p in m.pages:
            p[m.table[0, 25:].long()] = float("nan")  # the pages of the first sequence's drafts
        m2, p2 = gqa.gqa_tree_mask(i32(parents), indptr, full, max_tokens=20)
        got = m.tree(m.append(x, m.pages, full, indptr, p2), full, indptr, m2, p2)
        m.one(q[:3].contiguous(), m.pages, full)
        assert torch.equal(got, want)


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_starved_producers_time_out(cache):
    """Every wait expires after about 2 s, the call ends, its error is reported, and later calls are unaffected."""
    b = Batch([6, 30], [3000, 200], hq=8, hkv=2, page=64, dtype=BF16, cache=cache, seed=35)
    want = gqa.gqa_paged_tree_attn(**b.args())
    torch.cuda.synchronize()
    gqa.gqa_debug_starve_producers(True)
    try:
        gqa.gqa_paged_tree_attn(**b.args())
        torch.cuda.synchronize()
    finally:
        gqa.gqa_debug_starve_producers(False)
    assert gqa.gqa_check_device_errors(0) & 1
    assert torch.equal(gqa.gqa_paged_tree_attn(**b.args()), want)


def test_offsets_past_32_bits():
    """Caches of more than 2^31 elements: tree attention and compaction reach their last pages."""
    pages, hkv, page, d = 2 ** 31 // (8 * 64 * 128) + 40, 8, 64, 128
    k, v = (torch.zeros(pages, hkv, page, d, dtype=E4M3, device=DEV) for _ in range(2))
    small = Batch([10, 4], [300, 70], hq=16, hkv=8, page=64, dtype=BF16, cache=E4M3, seed=36)
    used = small.table.clamp(min=0).unique().long()
    for big, p in ((k, small.k), (v, small.v)):
        big[pages - 20 + used] = p[used]
    a = small.args()
    want = gqa.gqa_paged_tree_attn(**a)
    far = torch.where(small.table >= 0, small.table + pages - 20, small.table).to(torch.int32)
    assert torch.equal(gqa.gqa_paged_tree_attn(**{**a, "k_pages": k, "v_pages": v, "block_table": far}), want)
    kept, count = i32([[1, 3, 9], [2, 0, 0]]), i32([3, 1])
    small_pages = (small.k.contiguous(), small.v.contiguous())
    gqa.gqa_paged_keep(small_pages, small.table, a["qo_indptr"], a["kv_lens"], kept, count)
    gqa.gqa_paged_keep((k, v), far, a["qo_indptr"], a["kv_lens"], kept, count)
    for big, p in zip((k, v), small_pages):
        assert torch.equal(big[pages - 20 + used].view(torch.uint8), p[used].view(torch.uint8))
    assert not k[:pages - 40].view(torch.uint8).any()
