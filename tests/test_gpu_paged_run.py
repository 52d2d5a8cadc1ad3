"""GPU: the paged-cache operators together, as a serving loop runs them -- prompts
appended, then decode steps of append and attention, captured into graphs, on other
streams and from several threads."""
import threading

import pytest
import torch

import gqa_attention_kv_split_gb300 as gqa
import paged_reference as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


def rope_table(n, rot):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


class Server:
    """A batch of sequences over one cache, and the same on the CPU in 64 bits."""

    def __init__(self, B=5, hq=8, hkv=2, d=128, page=16, cap=256, dtype=torch.bfloat16, cache=None, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.B, self.hq, self.hkv, self.d, self.page, self.dtype = g, B, hq, hkv, d, page, dtype
        self.cache = cache or dtype
        mp = cap // page
        self.table = torch.randperm(B * mp, generator=g).to(torch.int32).view(B, mp)
        self.lens = torch.zeros(B, dtype=torch.int32)
        self.rope = rope_table(cap, d)
        self.scales = (0.02, 0.01) if self.cache == torch.float8_e4m3fn else (1.0, 1.0)
        shape = (B * mp, hkv, page, d)
        self.pages = [torch.full(shape, float("nan")).to(self.cache).to(DEV) for _ in range(2)]
        self.d_table, self.d_rope = self.table.to(DEV), self.rope.to(DEV)

    def new(self, q_lens):
        n = sum(q_lens)
        x = torch.randn(n, self.hq + 2 * self.hkv, self.d, generator=self.g).to(self.dtype)
        return x

    def split(self, x):
        return x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]

    def append(self, x, lens, indptr, **kw):
        q, k, v = self.split(x)
        return gqa.gqa_paged_append(q, k, v, *self.pages, self.d_table, lens, qo_indptr=indptr, rope=self.d_rope,
                                    k_scale=self.scales[0], v_scale=self.scales[1], **kw)

    def attend(self, q, lens, **kw):
        return gqa.gqa_paged_attn(q, *self.pages, self.d_table, lens, k_scale=self.scales[0], v_scale=self.scales[1], **kw)

    def check(self, q, out, lse, lens):
        """Against attention over what the cache now holds (the append has its own tests)."""
        pages = [torch.nan_to_num(p.float().cpu()).to(self.cache) for p in self.pages]
        R.check_attention(out, lse, q.cpu(), *pages, self.table, lens, k_scale=self.scales[0], v_scale=self.scales[1])


@pytest.mark.parametrize("dtype,cache", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16),
                                         (torch.bfloat16, torch.float8_e4m3fn)])
def test_prompts_then_decode_steps(dtype, cache):
    s = Server(dtype=dtype, cache=cache)
    prompts = [40, 1, 0, 17, 130]
    rows = s.new(prompts)
    history = {b: [] for b in range(s.B)}
    at = 0
    for b, n in enumerate(prompts):
        history[b] += [rows[at + i] for i in range(n)]
        at += n
    lens = torch.tensor(prompts, dtype=torch.int32)
    indptr = torch.tensor([0, 40, 41, 41, 58, 188], dtype=torch.int32, device=DEV)
    s.append(rows.to(DEV), lens.to(DEV), indptr)
    for step in range(4):
        lens = lens + 1
        x = s.new([1] * s.B)
        for b in range(s.B):
            history[b].append(x[b])
        q = s.append(x.to(DEV), lens.to(DEV), None)
        lse = torch.empty(s.B, s.hq, device=DEV)
        out = s.attend(q, lens.to(DEV), lse=lse)
        s.check(q, out, lse, lens)
    # and from the rows themselves, cache rounding and all left out: near the exact decode
    for b in range(s.B):
        h = torch.stack(history[b]).double()
        q, k, v = s.split(h)
        where = [(0, i) for i in range(len(h))]
        q, k = (R.rotated(t, s.rope, where, False) for t in (q, k))
        kk, vv = k.repeat_interleave(4, 1), v.repeat_interleave(4, 1)
        p = torch.softmax(torch.einsum("hd,thd->ht", q[-1], kk) / s.d ** 0.5, -1)
        want = torch.einsum("ht,thd->hd", p, vv)
        # inputs of the products rounded to the cache's type: half a step each of K (in the scores, about
        # |q||k| / sqrt(d) * eps / 2 in the mean square) and of V
        eps = 2.0 ** -4 if cache == torch.float8_e4m3fn else torch.finfo(dtype).eps / 2
        assert (out[b].cpu().double() - want).norm() <= 4 * eps * want.norm() + 2.0 ** -8 * want.norm()


def test_captured_step_follows_the_lengths():
    """One graph of append + attention, replayed as the sequences grow and end; the workspace comes from the graph's pool."""
    s = Server(B=6, cap=512, seed=1)
    prompts = [300, 5, 60, 1, 64, 120]
    lens = torch.tensor(prompts, dtype=torch.int32)
    indptr = torch.tensor([0] + list(torch.tensor(prompts).cumsum(0)), dtype=torch.int32, device=DEV)
    s.append(s.new(prompts).to(DEV), lens.to(DEV), indptr)
    x = torch.zeros(6, s.hq + 2 * s.hkv, s.d, dtype=s.dtype, device=DEV)
    d_lens = torch.zeros(6, dtype=torch.int32, device=DEV)
    lse = torch.empty(6, s.hq, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = s.append(x, d_lens, None)
        out = s.attend(q, d_lens, lse=lse)
    for step in range(5):
        lens = lens + 1
        if step == 3:
            lens[0] = 0  # a sequence has ended: its row is inactive
        lens[lens == 1] = 0 if step > 3 else 1
        x.copy_(s.new([1] * 6))
        q.zero_()
        d_lens.copy_(lens)
        graph.replay()
        torch.cuda.synchronize()
        s.check(q, out, lse, lens)
        lens[lens == 0] = -1 if step < 4 else 0
        lens = lens.clamp(min=0)


def test_two_graphs_replayed_at_once():
    """Two captured attentions, each with its own workspace, on two streams."""
    servers = [Server(B=3, hq=16, hkv=1, cap=4096, page=64, seed=2 + i) for i in range(2)]
    graphs, outs, args = [], [], []
    for s in servers:
        n = [4000, 77, 1000]
        lens = torch.tensor(n, dtype=torch.int32, device=DEV)
        q = s.append(s.new(n).to(DEV), lens, torch.tensor([0, 4000, 4077, 5077], dtype=torch.int32, device=DEV))
        q = q[[3999, 4076, 5076]].contiguous()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = s.attend(q, lens)
        graphs.append(g)
        outs.append(out)
        args.append((s, q, lens))
    want = [s.attend(q, lens).clone() for s, q, lens in args]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(50):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_workspace_of_the_caller_holds_anything():
    """A workspace needs no preparation: random bytes, another layout's leavings, the same graph twice."""
    a, b = Server(B=2, hq=16, hkv=1, cap=2048, page=64, seed=5), Server(B=3, hq=4, hkv=4, d=64, cap=2048, page=16, seed=6)
    ws = torch.randint(0, 256, (6 << 20,), dtype=torch.uint8, device=DEV)
    data = []
    for s in (a, b):
        n = [1500] * s.B
        lens = torch.tensor(n, dtype=torch.int32, device=DEV)
        indptr = torch.arange(0, 1500 * s.B + 1, 1500, dtype=torch.int32, device=DEV)
        q = s.append(s.new(n).to(DEV), lens, indptr)[1499::1500].contiguous()
        data.append((s, q, lens, s.attend(q, lens)))
    for _ in range(3):
        for s, q, lens, want in data:
            assert torch.equal(s.attend(q, lens, workspace=ws), want)
    s, q, lens, want = data[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.attend(q, lens, workspace=ws)
    for i in range(20):
        if i % 3 == 1:
            ws.random_(0, 256)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        t, tq, tl, tw = data[1]
        assert torch.equal(t.attend(tq, tl, workspace=ws), tw)


def test_captured_call_without_workspace_is_refused_by_the_library():
    """The entry point asks for one (the binding then takes it from the graph's pool); the library's own is not captured."""
    s = Server(B=2, seed=9)
    lens = torch.tensor([1, 1], dtype=torch.int32, device=DEV)
    q = s.append(s.new([1, 1]).to(DEV), lens, None)
    out = torch.empty_like(q)
    args = (q, *s.pages, s.d_table, lens, out, None, None, 1.0, 1.0, 1.0, 0, 0.0)
    assert gqa._binding().attn(*args) == 0
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens.add_(0)  # (a graph with something in it)
        status = gqa._binding().attn(*args)
    assert status == 7 and b"workspace of its own" in gqa.lib().gqa_last_error()
    gqa.gqa_release_workspace()
    again = s.attend(q, lens)
    torch.cuda.synchronize()
    assert torch.equal(again, out)


def test_threads_and_streams():
    """Calls from several threads, each on a stream of its own, give what one call gives."""
    s = Server(B=4, hq=16, hkv=2, cap=2048, page=32, seed=7)
    n = [2000, 3, 700, 64]
    lens = torch.tensor(n, dtype=torch.int32, device=DEV)
    q = s.append(s.new(n).to(DEV), lens, torch.tensor([0, 2000, 2003, 2703, 2767], dtype=torch.int32, device=DEV))
    q = q[[1999, 2002, 2702, 2766]].contiguous()
    want = s.attend(q, lens)
    torch.cuda.synchronize()
    bad = []

    def work():
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(30):
                if not torch.equal(s.attend(q, lens), want):
                    bad.append(1)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_threads_on_one_stream():
    """Calls of several threads on one stream share its workspace: no call's kernels come between another's two."""
    s = Server(B=3, hq=16, hkv=1, cap=4096, page=64, seed=12)
    batches = []
    for n in ([4000, 3, 900], [10, 3500, 2000], [1, 1, 4096], [2222, 2222, 2222]):
        lens = torch.tensor(n, dtype=torch.int32, device=DEV)
        q = torch.randn(3, 16, 128, device=DEV).bfloat16()
        batches.append((q, lens))
    full = torch.tensor([4096] * 3, dtype=torch.int32, device=DEV)
    s.append(s.new([4096] * 3).to(DEV), full, torch.tensor([0, 4096, 8192, 12288], dtype=torch.int32, device=DEV))
    want = [s.attend(*b) for b in batches]
    torch.cuda.synchronize()
    bad, stream, start = [], torch.cuda.Stream(), threading.Barrier(4)

    def work(i):
        with torch.cuda.stream(stream):
            out = torch.empty_like(want[i])
            start.wait(60)
            outs = [s.attend(*batches[i], out=out).clone() for _ in range(100)]
        stream.synchronize()
        if not all(torch.equal(o, want[i]) for o in outs):
            bad.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_nvfp4_chunked_prefill():
    """A prompt appended in two chunks and attended to chunk by chunk is the prompt appended and attended to at once."""
    g = torch.Generator().manual_seed(8)
    n, cut = 200, 96
    x = torch.randn(n, 48, 128, generator=g).bfloat16().to(DEV)
    q, k, v = x[:, :32], x[:, 32:40], x[:, 40:]
    rope = rope_table(n, 128).to(DEV)
    table = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device=DEV)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)

    def cache():
        z = lambda w: torch.zeros(4, 8, 64, w, dtype=torch.uint8, device=DEV)
        return z(64), z(8), z(64), z(8)

    one = cache()
    q8 = gqa.nvfp4_paged_append(q, k, v, *one, table, i32(0, n), i32(n), rope=rope, q_scale=0.02)
    want = gqa.nvfp4_paged_ctx_attn(q8, *one, table, i32(0, n), i32(n), q_scale=0.02, out_scale=2.0 ** -4)
    two, parts, q_parts = cache(), [], []
    for lo, hi in ((0, cut), (cut, n)):
        p8 = gqa.nvfp4_paged_append(q[lo:hi], k[lo:hi], v[lo:hi], *two, table, i32(0, hi - lo), i32(hi), rope=rope, q_scale=0.02)
        q_parts.append(p8)
        parts.append(gqa.nvfp4_paged_ctx_attn(p8, *two, table, i32(0, hi - lo), i32(hi), q_scale=0.02, out_scale=2.0 ** -4))
    assert torch.equal(torch.cat(q_parts), q8)
    for a, b in zip(one, two):
        assert torch.equal(a, b)
    val = lambda t: t.view(torch.float8_e4m3fn).float()
    # the same keys in other tiles: an output may round to the other neighbour
    got, ref = val(torch.cat(parts)), val(want)
    assert ((got - ref).abs() <= 2.0 ** -3 * ref.abs() + 2.0 ** -9).all()


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements: the last pages are written and read, their neighbours 2^31 elements before are not."""
    pages, hkv, page, d = 2 ** 31 // (8 * 64 * 128) + 40, 8, 64, 128
    cache = [torch.zeros(pages, hkv, page, d, dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    assert cache[0].numel() > 2 ** 31
    g = torch.Generator().manual_seed(10)
    n = 100
    x = torch.randn(n, 48, d, generator=g).bfloat16().to(DEV)
    q, k, v = x[:, :32], x[:, 32:40], x[:, 40:]
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    rope = rope_table(n, d).to(DEV)
    turned = gqa.gqa_paged_append(q, k, v, *cache, table, lens, qo_indptr=torch.tensor([0, n], dtype=torch.int32, device=DEV), rope=rope,
                                  k_scale=0.02, v_scale=0.02)
    last = turned[-1:].contiguous()
    lse = torch.empty(1, 32, device=DEV)
    out = gqa.gqa_paged_attn(last, *cache, table, lens, lse=lse, k_scale=0.02, v_scale=0.02)
    used = [pages - 1, pages - 3]
    small = [c[used].cpu() for c in cache]
    R.check_attention(out, lse, last.cpu(), *small, torch.tensor([[0, 1]]), lens.cpu(), k_scale=0.02, v_scale=0.02)
    for c in cache:
        written = (c.view(torch.uint8).flatten(1) != 0).any(1).nonzero().flatten().tolist()
        assert written == sorted(used)
    # the same rows in a small cache
    other = [torch.zeros(2, hkv, page, d, dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    gqa.gqa_paged_append(q, k, v, *other, torch.tensor([[0, 1]], dtype=torch.int32, device=DEV), lens,
                         qo_indptr=torch.tensor([0, n], dtype=torch.int32, device=DEV), rope=rope, k_scale=0.02, v_scale=0.02)
    for a, b in zip(other, small):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))


def test_first_calls_of_a_process_can_be_captured():
    """A fresh process whose first append and attention are captured ones."""
    import os
    import subprocess
    import sys
    code = """
import torch, gqa_attention_kv_split_gb300 as gqa
d = torch.device('cuda:0')
x = torch.randn(2, 6, 64, device=d).half()
pages = [torch.zeros(4, 1, 16, 64, dtype=torch.float16, device=d) for _ in range(2)]
table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=d)
lens = torch.tensor([1, 1], dtype=torch.int32, device=d)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    q = gqa.gqa_paged_append(x[:, :4], x[:, 4:5], x[:, 5:], *pages, table, lens)
    out = gqa.gqa_paged_attn(q, *pages, table, lens)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, x[:, 5:].expand(-1, 4, -1)), (out, x)
assert gqa.gqa_check_device_errors(0) == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_workspace_is_allocated_while_another_stream_is_captured():
    """The first eager call on a stream allocates its workspace without ending a capture that is going on."""
    s = Server(B=2, seed=11)
    lens = torch.tensor([1, 1], dtype=torch.int32, device=DEV)
    q = s.append(s.new([1, 1]).to(DEV), lens, None)
    out = torch.empty_like(q)
    want = s.attend(q, lens).clone()
    torch.cuda.synchronize()
    gqa.gqa_release_workspace()
    side, ready, done, bad = torch.cuda.Stream(), threading.Event(), threading.Event(), []

    def work():
        ready.wait(60)
        try:
            with torch.cuda.stream(side):
                s.attend(q, lens, out=out)
        except Exception as e:  # pragma: no cover
            bad.append(e)
        done.set()
    t = threading.Thread(target=work)
    t.start()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.attend(q, lens)
        ready.set()
        assert done.wait(60)
    t.join()
    graph.replay()
    torch.cuda.synchronize()
    assert not bad and torch.equal(got, want) and torch.equal(out, want)
